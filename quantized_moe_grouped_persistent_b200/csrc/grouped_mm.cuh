// grouped_mm.cuh -- sm_100a kernels of the grouped products (qgmm_mm.h).
//
//   mm_rows_kernel    out[i][j] = sum_c a[i][c] * W(g, c, j): the product (c = k, j = n) and
//                     the input gradient (c = n, j = k), 16-bit or MXFP4
//   mm_wgrad_kernel   dw[g][c][j] = sum_i a[i][c] * b[i][j] over the expert's rows
//   mm_join_kernel, mm_join_wgrad_kernel   add up the parts of sums that several pairs share
//   mm_sf_atoms_kernel                     arranges MXFP4 scale words for the tensor core
//
// The products are persistent on CTA pairs (tcgen05 cta_group::2, M = 256).  The weights' columns
// j take the M side and the rows i the N side, because N is what an instruction can
// choose freely: a group's rows are cut into tiles of equal height, rounded up to 16,
// so one row costs an N = 16 tile and no group pays for more than 15 rows of padding.
// The other way round, one row would cost as much as 128.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "groups.cuh"
#include "ptx_sm100.cuh"

namespace qgmm {

constexpr int MM_MAX_E = 1024;
constexpr int MM_M = 256;               // M of a pair's tile: 128 per CTA
constexpr int MM_STAGE_K = 128;         // bytes of the summed dimension per stage: one swizzle row
constexpr int MM_A_BYTES = 128 * MM_STAGE_K;
constexpr int MM_B_BYTES = 128 * MM_STAGE_K;
constexpr int MM_LOW_N = 64;            // greatest height of a low tile
constexpr int MM_LOW_B_BYTES = MM_LOW_N / 2 * MM_STAGE_K;
constexpr int MM_PANEL = 8;             // row tiles that share a sweep over the columns
constexpr int MM_TABLE_BYTES = (2 * (MM_MAX_E + 1) * 4 + 15) / 16 * 16;
constexpr int MM_EPI_WARPS = 4;         // one per quarter of the lanes
constexpr int MM_EPI_GROUPS = 2;        // mm_rows_kernel: groups of them, every second 32 rows each
constexpr int MM_OUT_ROWS = 16;         // rows of an output copy
constexpr int MM_OUT_PANEL = 32 * 128;  // staged 16-bit output: two panels of 32 rows x 64 columns
constexpr int MM_OUT_BYTES = 2 * MM_OUT_PANEL;
constexpr int MM_SF_ATOM = 512;         // scale words of 128 rows x 128 elements, as tcgen05.cp takes them

enum MmKind : int { MM_F16 = 0, MM_MXF4 = 1 };

// Stages whose products the tensor core adds up before the sum is taken out.  It truncates
// where f32 additions round, so a long sum drifts towards zero, by some 1.0e-9 of itself a term where
// signs are mixed and 6.0e-9 where all terms have one sign.  f32 outputs therefore leave the tensor
// core every 8 stages (512 terms) and are added up, rounded, in the epilogue's registers (0.7e-6 off in the
// norm at any length, one sign 2.5e-6).  MXFP4 products have few bits and mostly add up exactly;
// theirs leave every 32 stages (8192 terms), into memory, whose threads have no registers to
// spare (0.4e-6 with mixed signs and block scales 2^10 apart; 16-bit outputs stay to the end).
// 16-bit outputs, whose own rounding is 2.1e-4 in the norm (fp16; bf16 1.7e-3), stay to the end where
// the sum has MM_LONG_TERMS terms or fewer (0.9e-5 of drift, one sign 4.9e-5); longer ones (`LONG`)
// leave every 32 stages (2048 terms), into registers, since the drift would come to 0.7e-4 (one
// sign 3.9e-4) at 65536.  That costs 2% there (4 experts, 8192 rows, k = 16384, n = 2048, bf16: 399 us,
// whole 391) and more in shorter sums (32 experts, 32768 rows, k = 2048, n = 7168 in segments of
// 1024: 720 us, whole 692; 8 rows 43 and 38).
constexpr int MM_LONG_TERMS = 8192;
template <int KIND, typename O, bool LONG>
constexpr int MM_SEGMENT = KIND == MM_MXF4 ? (sizeof(O) == 2 ? 1 << 30 : 32) : sizeof(O) == 4 ? 8 : LONG ? 32 : 1 << 30;
// The same of the weight gradient, whose sums run over an expert's rows.  Where a call has rows for a
// second segment (`LONG`), 16-bit outputs leave the tensor core every 8192 rows (fp16) or 32768 (bf16;
// 0.3e-4 of drift, one sign 2.0e-4, of a rounding of 1.7e-3): the epilogue's threads keep their sums in the
// workspace until the last segment, since one group of them has no registers for 256 columns, and
// two were slower (launch_wgrad).  That kernel is some 2% slower for experts of one segment, too (32
// experts, 32768 rows, k = 2048, n = 7168, fp16: 850 us, whole 835; one of 300000 rows, k = n = 2048,
// bf16: 1994, whole 1984).
template <typename O>
constexpr int MM_LONG_SEGMENT = 512;
template <>
constexpr int MM_LONG_SEGMENT<__half> = 128;
template <typename O, bool LONG>
constexpr int MM_WGRAD_SEGMENT = sizeof(O) == 4 ? 8 : LONG ? MM_LONG_SEGMENT<O> : 1 << 30;
constexpr int64_t MM_KEPT_BYTES = 2 * 128 * 256 * 4;   // of a pair: f32 of its tile

struct MmArgs {
    const int64_t *group_list;
    int64_t m;
    int32_t e, group_list_type;
    int32_t c, j;              // rows: summed and output widths; wgrad: dw's rows and columns
    int32_t bf16;              // 16-bit operands: bf16 or fp16
    int32_t w_mn;              // rows: w's rows run along j (MN-major A tiles) instead of along c
    int32_t w_blocks;          // rows, w_mn: w's rows are whole blocks of 64 j, two of which come in one copy
    const uint8_t *sfa, *sfw;  // MXFP4: scales of a [m] and w [e, j], rows ld_sfa and ld_sfw bytes apart
    int64_t ld_sfa, ld_sfw;
    int32_t sf_bytes;          // widest aligned load of scales: 16, 4 or 1 bytes
    uint64_t cols_magic;       // rows: 2^40 over the column tiles, rounded up
    int32_t tile_n;            // rows: greatest height of a tile, MM_LOW_N or the kind's TILE_N
    int32_t splits, split_kb;  // parts of the sum, for mm_join_kernel (rows: of split_kb stages each); 1 = whole sums
    int64_t split_out;         // elements from one part's output to the next
    int32_t sf_atoms;          // the scale words come ready from mm_sf_atoms_kernel
    uint32_t *atoms_w, *atoms_a;
    void *out;
    int64_t ldo;               // row stride of out
    int64_t out_group;         // wgrad: group stride of dw
    int32_t accumulate;        // wgrad: add to dw
    float *kept;               // wgrad, 16-bit: MM_KEPT_BYTES a pair, where an expert may have rows for two segments
    int32_t stall_producer;    // test hook: no copy is issued, so every wait runs out
    uint32_t *status;
};

// Tensor maps of mm_rows_kernel.
struct MmRowsMaps {
    CUtensorMap w;         // 128 bytes x 128 rows (c fastest), or (j fastest) 64 j x 64 c, twice if MmArgs::w_blocks
    CUtensorMap a;         // 128 bytes x half the greatest tile's rows
    CUtensorMap low[4];    // 128 bytes x 64, 32, 16 and 8 rows
    CUtensorMap sfw, sfa;  // arranged scale words, 1 KB x 1 and x 2
    CUtensorMap out;       // 16-bit output, 64 columns x MM_OUT_ROWS
};

template <int KIND>
struct MmRowsCfg {
    // A ring of STAGES stages with half the greatest tile's rows of a each, or, where no tile
    // has more than MM_LOW_N rows, of LOW_STAGES with 32: calls with few rows are bound by how
    // many bytes of the weights are on their way.
    static constexpr int STAGES = 6;
    static constexpr int LOW_STAGES = KIND == MM_MXF4 ? 7 : 9;
    // 16-bit: two accumulators of 256 columns fill tensor memory.  MXFP4 keeps 64 columns
    // for two stages' scale words, so its tiles have 224 rows at most.
    static constexpr int TILE_N = KIND == MM_MXF4 ? 224 : 256;
    static constexpr int B_BYTES = TILE_N / 2 * MM_STAGE_K;
    static constexpr int SF_WARPS = KIND == MM_MXF4 ? 4 : 0;
    static constexpr int EPI_WARPS = MM_EPI_GROUPS * MM_EPI_WARPS;
    static constexpr int THREADS = (2 + EPI_WARPS + SF_WARPS) * 32;
    static constexpr int SF_BYTES = KIND == MM_MXF4 ? 6 * MM_SF_ATOM : 0;   // w: 2 atoms, rows: 2 x 2
    static constexpr int NUM_BARS = 2 * LOW_STAGES + 2 + 2 + 1;
    static constexpr int CTRL_BYTES = (NUM_BARS * 8 + 16 + 15) / 16 * 16;
    static constexpr size_t RING = size_t(STAGES) * (MM_A_BYTES + B_BYTES + SF_BYTES);
    static constexpr size_t OFF_OUT = RING;   // per epilogue group, 32 output rows
    static constexpr size_t OFF_CTRL = OFF_OUT + MM_EPI_GROUPS * MM_OUT_BYTES;
    static_assert(OFF_OUT % 1024 == 0, "the swizzle counts from 1 KB");
    static_assert(LOW_STAGES * (MM_A_BYTES + MM_LOW_B_BYTES + SF_BYTES) <= RING, "the low ring fits the other's room");
    static constexpr size_t OFF_TABLE = OFF_CTRL + CTRL_BYTES;
    static constexpr size_t SMEM_BYTES = 1024 + OFF_TABLE + MM_TABLE_BYTES;
    static_assert(SMEM_BYTES <= 232448, "shared memory above the sm_100 per-block limit");
};

// GROUPS of four epilogue warps, each warp with its 4 KB of staging: a second group empties
// tiles faster and leaves room for a stage less.
template <int GROUPS>
struct MmWgradCfg {
    static constexpr int STAGES = GROUPS == 1 ? 6 : 5;
    static constexpr int EPI_WARPS = GROUPS * MM_EPI_WARPS;
    static constexpr int THREADS = (2 + EPI_WARPS + 1) * 32;   // the last warp clears rows past a group's end
    static constexpr int NUM_BARS = 3 * STAGES + 2 + 2 + 1;
    static constexpr int CTRL_BYTES = (NUM_BARS * 8 + 16 + 15) / 16 * 16;
    static constexpr int STAGING = EPI_WARPS * 32 * 128;          // per epilogue warp 32 rows x 128 bytes
    static constexpr size_t OFF_STAGING = size_t(STAGES) * (MM_A_BYTES + MM_B_BYTES);
    static constexpr size_t OFF_CTRL = OFF_STAGING + STAGING;
    static constexpr size_t OFF_TABLE = OFF_CTRL + CTRL_BYTES;
    static constexpr size_t SMEM_BYTES = 1024 + OFF_TABLE + MM_TABLE_BYTES;
    static_assert(SMEM_BYTES <= 232448, "shared memory above the sm_100 per-block limit");
};

// ---------------------------------------------------------------- small parts
__device__ __forceinline__ uint32_t mm_pack2(const __nv_bfloat16 *, float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t mm_pack2(const __half *, float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 mm_unpack2(const __nv_bfloat16 *, uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float2 mm_unpack2(const __half *, uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// Where tile `t` of an expert's dw lies: `tiles` row tiles by `cols` column tiles in panels
// of MM_PANEL row tiles, the row tile fastest.
__device__ __forceinline__ void mm_panel(int t, int tiles, int cols, int &row_tile, int &col_tile)
{
    const int p = t / (MM_PANEL * cols);
    const int left = tiles - p * MM_PANEL;
    const int high = left < MM_PANEL ? left : MM_PANEL;
    const int r = t - p * MM_PANEL * cols;
    col_tile = r / high;
    row_tile = p * MM_PANEL + (r - col_tile * high);
}

// Pairs that take tiles: with the rounds that all of them need anyway, as few as share them
// evenly.  A last round that a few pairs run alone is bound by latency, while the fewer pairs
// still take all of the memory's bandwidth (224 tiles of 1 MB on 74 pairs: 43.7 us, on 56: 39.5).
__device__ __forceinline__ int mm_active_pairs(int tiles, int pairs)
{
    const int rounds = (tiles + pairs - 1) / pairs;
    return rounds ? (tiles + rounds - 1) / rounds : pairs;
}

struct MmTile {
    int g, mt;           // expert, and row tile of the whole walk
    int row0, rows;      // first row and row count
    int n;               // the instruction's N: rows rounded up to 16
    int j0;
};

// The walk over a call's tiles, expert by expert.  Every warp's walk goes up, so a look at the
// expert of its last tile mostly finds the next one's, and the divisions are by factors fixed
// for the call: a tile's place costs some 100 cycles instead of 700, which a warp that issues
// instructions cannot hide behind a short sum (MXFP4 at m = 32768, k = 2048, n = 7168: 304 us
// before, 298 so).
struct MmWalk {
    const int32_t *off, *cum;
    int e, cols, g;
    uint64_t magic;      // t / cols = t * magic >> 40, exact below 2^40 / cols (t stays below 2^27)

    __device__ __forceinline__ MmWalk(const int32_t *off_, const int32_t *cum_, int e_, int cols_, uint64_t magic_)
        : off(off_), cum(cum_), e(e_), cols(cols_), g(0), magic(magic_)
    {
    }

    __device__ __forceinline__ int by_cols(int t) const
    {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(t)) * magic) >> 40);
    }

    __device__ __forceinline__ MmTile at(int t)
    {
        if (t >= cum[g + 1] * cols || t < cum[g] * cols) {
            const int mt = by_cols(t);
            int lo = 0, hi = e;   // cum[lo] <= mt < cum[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cum[mid] <= mt) lo = mid;
                else hi = mid;
            }
            g = lo;
        }
        MmTile c;
        c.g = g;
        const int first = cum[g], tiles = cum[g + 1] - first, rows = off[g + 1] - off[g];
        // panels of MM_PANEL row tiles, the row tile fastest, so that the pairs at work share
        // both operands in L2 however large the weights are
        const int r = t - first * cols;
        const int p = by_cols(r) / MM_PANEL;
        const int high = tiles - p * MM_PANEL < MM_PANEL ? tiles - p * MM_PANEL : MM_PANEL;
        const int q = r - p * MM_PANEL * cols;         // below 8 * 256, so the float quotient is exact
        const float part = __frcp_rn(static_cast<float>(high));
        const int jt = high == MM_PANEL ? q / MM_PANEL : static_cast<int>((static_cast<float>(q) + 0.5f) * part);
        const int i = p * MM_PANEL + (q - jt * high);
        // equal heights, a multiple of 16: never above the greatest, and (tiles - 1) * height < rows
        const uint32_t even = static_cast<uint32_t>(rows + tiles - 1) / static_cast<uint32_t>(tiles);
        const int height = (static_cast<int>(even) + 15) & ~15;
        c.mt = first + i;
        c.row0 = off[g] + i * height;
        c.rows = rows - i * height < height ? rows - i * height : height;
        c.n = (c.rows + 15) & ~15;
        c.j0 = jt * MM_M;
        return c;
    }
};

// ---------------------------------------------------------------- out = a W
// Each CTA of a pair copies half of a tile's rows in the lowest box that holds them.  (Boxes
// that together hold them exactly were slower, for all the bytes saved: the number of copies
// counts.  A fourth to sixth copy a stage in every fourth tile: 692 us for 639.)
template <int KIND, typename O, bool LONG>
__global__ void __launch_bounds__(MmRowsCfg<KIND>::THREADS, 1)
    mm_rows_kernel(const __grid_constant__ MmRowsMaps maps, const MmArgs args)
{
    using Cfg = MmRowsCfg<KIND>;
    const bool low = args.tile_n <= MM_LOW_N;
    const int S = low ? Cfg::LOW_STAGES : Cfg::STAGES;
    const int b_slot = low ? MM_LOW_B_BYTES : Cfg::B_BYTES;
    constexpr int KE = KIND == MM_MXF4 ? 2 * MM_STAGE_K : MM_STAGE_K / 2;   // summed elements per stage
    constexpr int KI = KIND == MM_MXF4 ? 64 : 16;                           // and per instruction (32 bytes)
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *smem_w = smem;
    uint8_t *smem_a = smem + S * MM_A_BYTES;
    uint8_t *smem_sf = smem_a + S * b_slot;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_CTRL);
    uint64_t *full = bars;            // leader: both CTAs' operands landed
    uint64_t *empty = bars + Cfg::LOW_STAGES;       // both: the pair's MMAs finished reading the stage
    uint64_t *tfull = bars + 2 * Cfg::LOW_STAGES;   // both: accumulator ready
    uint64_t *tempty = tfull + 2;     // leader: both CTAs' epilogues drained it
    uint64_t *drain = tempty + 2;     // leader: all issued MMAs completed
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + Cfg::NUM_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int32_t *off = reinterpret_cast<int32_t *>(smem + Cfg::OFF_TABLE);
    int32_t *cum = off + (MM_MAX_E + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            // the producer, and both CTAs' scale warps where they write the scale words
            ptx::mbar_init(&full[s], KIND == MM_MXF4 && !args.sf_atoms ? 1 + 2 * Cfg::SF_WARPS : 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&tfull[b], 1);
            ptx::mbar_init(&tempty[b], 2 * Cfg::EPI_WARPS);
        }
        ptx::mbar_init(drain, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0) {
        ptx::pdl_wait_primary();   // what earlier kernels wrote is there for the whole block from the sync below on
        const uint32_t flags = decode_groups_warp(
            args.group_list, args.e, args.group_list_type, args.m,
            [=](int64_t rows) { return static_cast<int32_t>((rows + args.tile_n - 1) / args.tile_n); }, off, cum);
        if (lane == 0) {
            if (blockIdx.x == 0) {
                args.status[0] = flags;
                args.status[1] = static_cast<uint32_t>(off[args.e]);   // rows, for mm_join_kernel
            }
            ptx::prefetch_tmap(&maps.w);
            ptx::prefetch_tmap(low ? &maps.low[3] : &maps.a);
            if (sizeof(O) == 2) ptx::prefetch_tmap(&maps.out);
            if (KIND == MM_MXF4 && args.sf_atoms) {
                ptx::prefetch_tmap(&maps.sfw);
                ptx::prefetch_tmap(&maps.sfa);
            }
        }
    } else if (warp == 1) {
        ptx::tmem_alloc_pair(tmem_holder, 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();   // both CTAs' barriers are initialised before any copy or remote arrive
    ptx::tc_fence_after();
    ptx::pdl_launch_dependents();
    const uint32_t tmem_base = *tmem_holder;

    const int cols = (args.j + MM_M - 1) / MM_M;
    const int T = cum[args.e] * cols * (sizeof(O) == 4 ? args.splits : 1);
    const int nclusters = mm_active_pairs(T, gridDim.x >> 1);
    const int cluster = static_cast<int>(blockIdx.x >> 1) < nclusters ? blockIdx.x >> 1 : T;   // first tile, or none
    const int KB = (args.c + KE - 1) / KE;
    MmWalk walk(off, cum, args.e, cols, args.cols_magic);
    // tile t / splits, and its stages of part t % splits (parts are f32)
    constexpr bool SPLITS = sizeof(O) == 4;
    int kb0 = 0, kb1 = KB, part = 0;
    auto tile_at = [&](int t) {
        if (SPLITS && args.splits > 1) {
            const int whole = t / args.splits;
            part = t - whole * args.splits;
            kb0 = part * args.split_kb;
            kb1 = kb0 + args.split_kb < KB ? kb0 + args.split_kb : KB;
            t = whole;
        }
        return walk.at(t);
    };

    const bool atoms = KIND == MM_MXF4 && args.sf_atoms;
    const uint32_t full_leader0 = ptx::map_to_rank(&full[0], 0);

    auto fail = [&]() {
        atomicOr(args.status, QGMM_DEV_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp == 0) {
        // ------------------------------------------------ copies (both CTAs, own halves)
        // (One elected lane, as for the MMAs below: chosen by elect.sync, not by its number, it
        // keeps what the instructions take in uniform registers.)
        if (ptx::elect_one()) {
            uint32_t issued = 0;      // stages handed out: the last of each is waited for after a failure
            int stage = 0;
            uint32_t phase = 0;
            bool ok = args.stall_producer == 0;
            for (int t = cluster; t < T && ok; t += nclusters) {
                const MmTile c = tile_at(t);
                const int half = c.n / 2;
                const int row = c.row0 + half * static_cast<int>(rank);
                const int j = c.j0 + 128 * static_cast<int>(rank);
                const int box = half > 64 ? -1 : half > 32 ? 0 : half > 16 ? 1 : half > 8 ? 2 : 3;
                const CUtensorMap *map_a = box < 0 ? &maps.a : &maps.low[box];
                const uint32_t b_bytes = box < 0 ? Cfg::B_BYTES : (64 >> box) * MM_STAGE_K;
                const uint32_t tx = 2u * (MM_A_BYTES + b_bytes + (atoms ? Cfg::SF_BYTES : 0));
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!ptx::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
                        fail();
                        ok = false;
                        break;
                    }
                    if (leader) ptx::mbar_arrive_expect_tx(&full[stage], tx);
                    const uint32_t fb = full_leader0 + stage * 8u;
                    uint8_t *dw = smem_w + stage * MM_A_BYTES, *da = smem_a + stage * b_slot;
                    const int x = kb * (KIND == MM_MXF4 ? MM_STAGE_K : KE);   // MXFP4 maps count bytes
                    if (args.w_blocks) {
                        ptx::tma_load_4d_pair(dw, &maps.w, fb, 0, kb * KE, j / 64, c.g);
                    } else if (args.w_mn) {
                        ptx::tma_load_3d_pair(dw, &maps.w, fb, j, kb * KE, c.g);
                        ptx::tma_load_3d_pair(dw + MM_A_BYTES / 2, &maps.w, fb, j + 64, kb * KE, c.g);
                    } else {
                        ptx::tma_load_3d_pair(dw, &maps.w, fb, x, j, c.g);
                    }
                    ptx::tma_load_2d_pair(da, map_a, fb, x, row);
                    ++issued;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && leader) {
                // let the copies already in flight land before the CTA leaves
                for (uint32_t s = 0; s < static_cast<uint32_t>(S); ++s) {
                    if (issued <= s) continue;
                    volatile int never = 0;
                    ptx::mbar_wait(&full[s], ((issued - 1u - s) / S) & 1u, &never);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issue (leader CTA only)
        // A stage's four instructions go out without a loop, the next stage's barrier having
        // been looked at before them.
        if (leader && ptx::elect_one()) {
            // A tile in j-fastest layout: 64 j x 64 c atoms, 8 c rows 1 KB apart, j atoms 8 KB apart
            const uint32_t a_step = args.w_mn ? 16 * 128 : 32, a_lbo = args.w_mn ? MM_A_BYTES / 2 : 16;
            const uint64_t a_base = ptx::smem_desc_sw128(ptx::smem_addr(smem_w), a_lbo, 1024);
            const uint64_t b_base = ptx::smem_desc_sw128(ptx::smem_addr(smem_a), 16, 1024);
            int stage = 0;
            uint32_t phase = 0, sf_buf = 0;
            int lt = 0;
            bool ok = true;
            for (int t = cluster; t < T && ok; t += nclusters) {
                const MmTile c = tile_at(t);
                const uint32_t idesc = KIND == MM_MXF4 ? ptx::idesc_mxf4(MM_M, c.n, 0)
                                                       : ptx::idesc_f16(MM_M, c.n, args.bf16, args.w_mn, false);
                int buf = 0;
                uint32_t d_tmem = 0;
                bool ready = false;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const bool first = (kb - kb0) % MM_SEGMENT<KIND, O, LONG> == 0;
                    const bool last = kb + 1 == kb1 || (kb + 1 - kb0) % MM_SEGMENT<KIND, O, LONG> == 0;
                    if (first) {
                        buf = lt & 1;
                        const uint32_t use = static_cast<uint32_t>(lt >> 1) & 1u;
                        ++lt;
                        if (!ptx::mbar_wait(&tempty[buf], use ^ 1u, abort_flag)) {
                            fail();
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        d_tmem = tmem_base + static_cast<uint32_t>(buf * Cfg::TILE_N);
                        ready = ptx::mbar_test_wait_cluster(ptx::smem_addr(&full[stage]), phase);
                    }
                    if (!ready && !ptx::mbar_wait<KIND == MM_MXF4>(&full[stage], phase, abort_flag)) {
                        fail();
                        ok = false;
                        break;
                    }
                    const int next = stage + 1 == S ? 0 : stage + 1;
                    const uint32_t next_phase = next ? phase : phase ^ 1u;
                    ready = ptx::mbar_test_wait_cluster(ptx::smem_addr(&full[next]), next_phase);
                    const uint64_t a0 = a_base + stage * (MM_A_BYTES / 16), b0 = b_base + stage * (b_slot / 16);
                    uint32_t sfw_t = 0, sfa_t = 0;
                    if constexpr (KIND == MM_MXF4) {
                        // scale words: w's two 128-element halves, then each half's of the rows (2 x 128)
                        sfw_t = tmem_base + 2 * Cfg::TILE_N + 24u * sf_buf;
                        sfa_t = sfw_t + 8u;
                        sf_buf ^= 1u;
                        const uint64_t sf =
                            ptx::smem_desc_noswizzle(ptx::smem_addr(smem_sf + stage * Cfg::SF_BYTES), 16, 128);
#pragma unroll
                        for (int i = 0; i < 6; ++i) {   // atom i: block i / 2 (w, rows 0-127, 128-255), half i % 2
                            const uint32_t to = i < 2 ? 4u * i : 8u + 8u * (i & 1) + 4u * (i / 2 - 1);
                            if (i < 4 || c.n > 128)
                                ptx::tmem_cp_32x128b_warpx4_pair(sfw_t + to, sf + i * (MM_SF_ATOM / 16));
                        }
                    }
                    // past c both tiles hold zeros, so the last stage needs no shorter form
#pragma unroll
                    for (int kk = 0; kk < KE / KI; ++kk) {
                        const uint64_t adesc = a0 + kk * (a_step / 16), bdesc = b0 + kk * 2;
                        const uint32_t acc = kk ? 1u : !first;
                        if constexpr (KIND == MM_MXF4)
                            ptx::mma_mxf4_pair(d_tmem, adesc, bdesc, idesc | ptx::idesc_mxf4(0, 0, kk & 1),
                                               sfw_t + 4u * (kk >> 1), sfa_t + 8u * (kk >> 1), acc);
                        else
                            ptx::mma_f16_pair(d_tmem, adesc, bdesc, idesc, acc);
                    }
                    ptx::mma_commit_pair_both(&empty[stage]);
                    if (last) ptx::mma_commit_pair_both(&tfull[buf]);
                    stage = next;
                    phase = next_phase;
                }
            }
            ptx::mma_commit_pair(ptx::map_to_rank(drain, 0));
            volatile int never = 0;
            ptx::mbar_wait(drain, 0, &never);
        }
        __syncwarp();
    } else if (warp < 2 + Cfg::EPI_WARPS) {
        // ------------------------------------------------ epilogue (both CTAs, own 128 columns j)
        // A thread has one j and a chunk's 32 rows.  f32: a warp stores 128 contiguous bytes
        // per row.  16 bits: neighbouring lanes trade halves, so that each has two j of every
        // second row; the group's four warps gather 32 rows in shared memory, two panels of 64
        // columns in the 128-byte swizzle, and tile copies of 16 rows take them out.
        const int q = warp & 3, group = (warp - 2) / MM_EPI_WARPS;
        uint8_t *stage_mem = smem + Cfg::OFF_OUT + group * MM_OUT_BYTES;
        uint32_t tempty_leader[2];
        tempty_leader[0] = ptx::map_to_rank(&tempty[0], 0);
        tempty_leader[1] = ptx::map_to_rank(&tempty[1], 0);
        int lt = 0;
        bool ok = true;
        for (int t = cluster; t < T && ok; t += nclusters) {
            const MmTile c = tile_at(t);
            const int jc = c.j0 + 128 * static_cast<int>(rank);   // this CTA's columns: from jc up to j_end
            const int j_end = jc + 128 < args.j ? jc + 128 : args.j;
            const int j = jc + 32 * q + lane;
            O *const out = static_cast<O *>(args.out) + (SPLITS ? part * args.split_out : 0);
            constexpr bool IN_REGISTERS = KIND == MM_F16 && (sizeof(O) == 4 || LONG);
            constexpr int PARTS = Cfg::TILE_N / (32 * MM_EPI_GROUPS);   // parts of 32 rows of a group (16-bit kinds)
            float sum[IN_REGISTERS ? PARTS : 1][32];
            // 16-bit outputs: 32 rows of the tile from r0, by the whole group
            auto put16 = [&](int r0, const auto &v) {
                const int rows = c.rows - r0;
                if (lane == 0) ptx::bulk_wait_read<0>();   // the copies out of the group's buffer are through
                ptx::named_sync(1 + group, MM_EPI_WARPS * 32);
                const int odd = lane & 1, at = 32 * (q & 1) + lane - odd;   // column in the panel
                uint8_t *panel = stage_mem + (q >> 1) * MM_OUT_PANEL;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = (i & 3) | (i & 12) << 1;   // rows r and r + 4: 64 bytes of each, in other banks
                    const uint32_t mine = mm_pack2(static_cast<O *>(nullptr), v[r], v[r + 4]);
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
                    const int row = r + 4 * odd;
                    uint8_t *to = panel + row * 128 + (((at >> 3) ^ (row & 7)) << 4) + (at & 7) * 2;
                    *reinterpret_cast<uint32_t *>(to) =
                        odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
                }
                ptx::fence_async_shared();
                ptx::named_sync(1 + group, MM_EPI_WARPS * 32);
                const int copied = (rows < 32 ? rows : 32) & ~(MM_OUT_ROWS - 1);
                // four copies, one for each warp: a panel, and its first or second 16 rows
                const int x = jc + 64 * (q & 1), y = MM_OUT_ROWS * (q >> 1);
                if (lane == 0 && y < copied && x < j_end) {
                    ptx::tma_store_2d(&maps.out, stage_mem + (q & 1) * MM_OUT_PANEL + y * 128, x, c.row0 + r0 + y);
                    ptx::bulk_commit();
                }
                // a tile's last rows, which a copy would run past: 16 bytes a thread
                const int left = (rows < 32 ? rows : 32) - copied;
                for (int i = 32 * q + lane; i < 16 * left; i += 32 * MM_EPI_WARPS) {
                    const int row = copied + (i >> 4), piece = i & 15;
                    if (jc + 8 * piece < j_end)
                        *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(c.row0 + r0 + row) * args.ldo + jc + 8 * piece) =
                            *reinterpret_cast<const uint4 *>(stage_mem + (piece >> 3) * MM_OUT_PANEL + row * 128 +
                                                             (((piece & 7) ^ (row & 7)) << 4));
                }
            };
            for (int kb = 0; kb < kb1 - kb0; kb += MM_SEGMENT<KIND, O, LONG>, ++lt) {
                const int buf = lt & 1;
                const uint32_t use = static_cast<uint32_t>(lt >> 1) & 1u;
                // the warps share barriers below: they leave together or not at all
                if (!ptx::named_all(1 + group, MM_EPI_WARPS * 32, ptx::mbar_wait(&tfull[buf], use, abort_flag))) {
                    fail();
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t acc =
                    tmem_base + static_cast<uint32_t>(buf * Cfg::TILE_N) + (static_cast<uint32_t>(32 * q) << 16);
                if constexpr (IN_REGISTERS) {
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        const int r0 = 32 * (group + MM_EPI_GROUPS * i);
                        if (r0 >= c.rows) break;
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            uint32_t v[16];
                            ptx::tmem_ld_32x32b_x16(acc + r0 + h, v);
                            ptx::tmem_ld_wait(v);
#pragma unroll
                            for (int r = 0; r < 16; ++r) sum[i][h + r] = (kb ? sum[i][h + r] : 0.f) + __uint_as_float(v[r]);
                        }
                    }
                }
                for (int r0 = 32 * group; !IN_REGISTERS && r0 < c.rows; r0 += 32 * MM_EPI_GROUPS) {
                    float v[32];
                    {
                        uint32_t bits[32];
                        ptx::tmem_ld_32x32b_x32(acc + r0, bits);   // past N: columns of this CTA's allocation, unused
                        ptx::tmem_ld_wait(bits);
#pragma unroll
                        for (int r = 0; r < 32; ++r) v[r] = __uint_as_float(bits[r]);
                    }
                    if constexpr (sizeof(O) == 4) {
                        const int rows = c.rows - r0;
                        O *p = out + static_cast<int64_t>(c.row0 + r0) * args.ldo + j;
                        if (j < j_end) {
                            if (kb) {   // this thread's own stores of the segments before
                                float old[32];
#pragma unroll
                                for (int r = 0; r < 32; ++r) old[r] = r < rows ? p[r * args.ldo] : 0.f;
#pragma unroll
                                for (int r = 0; r < 32; ++r) v[r] += old[r];
                            }
#pragma unroll
                            for (int r = 0; r < 32; ++r)
                                if (r < rows) p[r * args.ldo] = v[r];
                        }
                    } else {
                        put16(r0, v);
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(tempty_leader[buf]);
            }
            if constexpr (IN_REGISTERS) {
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
                    const int r0 = 32 * (group + MM_EPI_GROUPS * i), rows = c.rows - r0;
                    if constexpr (sizeof(O) == 4) {
                        O *p = out + static_cast<int64_t>(c.row0 + r0) * args.ldo + j;
#pragma unroll
                        for (int r = 0; r < 32; ++r)
                            if (ok && r < rows && j < j_end) p[r * args.ldo] = sum[i][r];
                    } else if (ok && rows > 0) {
                        put16(r0, sum[i]);
                    }
                }
            }
        }
        if (lane == 0) ptx::bulk_wait_all();
        __syncwarp();
    } else if constexpr (KIND == MM_MXF4) {
        // ------------------------------------------------ scale words (both CTAs)
        // A stage's scale words, arranged as tcgen05.cp wants them: 512-byte atoms of 128
        // rows x 4 scales, row r's word at (r % 32) * 4 + r / 32.  Thread i * 4 + u takes row
        // i + 32 u of each operand, so a warp writes 128 consecutive bytes.  This CTA's
        // tensor memory needs its own 128 columns j and all of the tile's rows.
        const int st = threadIdx.x - (2 + Cfg::EPI_WARPS) * 32;
        const int r = (st >> 2) + 32 * (st & 3);
        const int blocks = args.c / 32;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        if (atoms) {
            // they come ready: the first of these warps copies them, beside warp 0's copies
            if (warp == 2 + Cfg::EPI_WARPS && ptx::elect_one()) {
                ok = args.stall_producer == 0;
                for (int t = cluster; t < T && ok; t += nclusters) {
                    const MmTile c = tile_at(t);
                    const int w0 = (c.g * 2 * cols + c.j0 / 128 + static_cast<int>(rank)) * KB;
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!ptx::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
                            fail();
                            ok = false;
                            break;
                        }
                        uint8_t *sf = smem_sf + stage * Cfg::SF_BYTES;
                        ptx::tma_load_2d_pair(sf, &maps.sfw, full_leader0 + stage * 8u, 0, w0 + kb);
                        ptx::tma_load_2d_pair(sf + 2 * MM_SF_ATOM, &maps.sfa, full_leader0 + stage * 8u, 0,
                                              (c.mt * KB + kb) * 2);
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            __syncwarp();
        }
        // The 16 scales of two stages from block b of a row, by the widest loads that k and
        // the strides allow (args.sf_bytes; where it is 1 they come ready).  Blocks past the
        // row's end get 2^-127: finite, against the zeros that the operands' tiles hold there.
        auto load16 = [&](const uint8_t *row, int b) -> uint4 {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (row && args.sf_bytes == 16) {
                if (b < blocks) return *reinterpret_cast<const uint4 *>(row + b);
            } else if (row) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (b + 4 * u < blocks) w[u] = *reinterpret_cast<const uint32_t *>(row + b + 4 * u);
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        // The stream of the walk's scales in pieces of four stages, AHEAD of them loaded before
        // the first is handed on: a load takes several stages' time when the copies are busy.
        constexpr int AHEAD = 3, PIECE = 4;
        struct Piece {
            uint4 v[3][PIECE / 2];   // w's row, rows r and 128 + r: 16 scales for each two stages
            int n;                   // stages; 0 ends the stream
        };
        Piece pieces[AHEAD];
        int next_t = atoms ? T : cluster, next_kb = 0;
        bool next_tile = true;
        const uint8_t *row[3] = {nullptr, nullptr, nullptr};
        auto fetch = [&](Piece &p) {
            p.n = 0;
            if (next_t >= T) return;
            if (next_tile) {
                const MmTile c = tile_at(next_t);
                next_kb = kb0;
                next_tile = false;
                const int j = c.j0 + 128 * static_cast<int>(rank) + r;
                row[0] = j < args.j ? args.sfw + (static_cast<int64_t>(c.g) * args.j + j) * args.ld_sfw : nullptr;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    row[1 + i] = 128 * i + r < c.rows
                                     ? args.sfa + static_cast<int64_t>(c.row0 + 128 * i + r) * args.ld_sfa
                                     : nullptr;
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int u = 0; u < PIECE / 2; ++u) p.v[i][u] = load16(row[i], 8 * next_kb + 16 * u);
            p.n = kb1 - next_kb < PIECE ? kb1 - next_kb : PIECE;
            next_kb += PIECE;
            if (next_kb >= kb1) {
                next_tile = true;
                next_t += nclusters;
            }
        };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) fetch(pieces[d]);
        while (ok && pieces[0].n) {
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                Piece &p = pieces[d];
#pragma unroll
                for (int h = 0; h < PIECE; ++h) {
                    if (!ok || h >= p.n) break;
                    if (!ptx::mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag)) {
                        fail();
                        ok = false;
                        break;
                    }
                    uint32_t *sf = reinterpret_cast<uint32_t *>(smem_sf + stage * Cfg::SF_BYTES) + st;
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        const uint4 v = p.v[i][h / 2];
                        sf[2 * i * (MM_SF_ATOM / 4)] = h & 1 ? v.z : v.x;
                        sf[(2 * i + 1) * (MM_SF_ATOM / 4)] = h & 1 ? v.w : v.y;
                    }
                    ptx::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster_release_smem(full_leader0 + stage * 8u);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                fetch(p);
            }
        }
    }

    ptx::tc_fence_before();
    ptx::cluster_sync();   // no remote arrive or pair MMA still targets either CTA
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, 512);
    }
}

// ---------------------------------------------------------------- MXFP4 scale words, arranged
// For calls with many rows: every stage's scale words as mm_rows_kernel's copies take them,
// once per call, since otherwise each tile gathers them anew, 16 bytes of a row at a time
// (at m = 32768, k = 2048, n = 7168 that cost the kernel 75 us of 390, at k = 8192 40%).
// One block of threads per 128 rows of w (or of a row tile): 1 KB per 256 elements, w's at
// (expert * 2 * tiles + block) * KB + kb, a row tile's at ((tile * KB) + kb) * 2 + block.
__global__ void __launch_bounds__(256) mm_sf_atoms_kernel(const MmArgs args)
{
    __shared__ int32_t off[MM_MAX_E + 1], cum[MM_MAX_E + 1];
    __shared__ uint32_t words[128][33];
    ptx::pdl_wait_primary();
    ptx::pdl_launch_dependents();
    if (threadIdx.x < 32)
        decode_groups_warp(
            args.group_list, args.e, args.group_list_type, args.m,
            [=](int64_t rows) { return static_cast<int32_t>((rows + args.tile_n - 1) / args.tile_n); }, off, cum);
    __syncthreads();
    const int cols = (args.j + MM_M - 1) / MM_M, blocks = args.c / 32;
    const int KB = (args.c + 2 * MM_STAGE_K - 1) / (2 * MM_STAGE_K);
    MmWalk walk(off, cum, args.e, 1, uint64_t(1) << 40);
    const int64_t units_w = int64_t(args.e) * 2 * cols, units = units_w + 2 * int64_t(cum[args.e]);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const uint8_t *src;
        int64_t ld;
        int rows, step;      // rows of the block; words from one stage to the next of dst
        uint32_t *dst;
        if (u < units_w) {
            const int g = static_cast<int>(u / (2 * cols)), block = static_cast<int>(u % (2 * cols));
            if (off[g] == off[g + 1]) continue;
            rows = args.j - 128 * block;
            ld = args.ld_sfw;
            src = args.sfw + (int64_t(g) * args.j + 128 * block) * ld;
            dst = args.atoms_w + u * KB * (2 * MM_SF_ATOM / 4);
            step = 2 * MM_SF_ATOM / 4;
        } else {
            const int mt = static_cast<int>((u - units_w) >> 1), block = static_cast<int>((u - units_w) & 1);
            const MmTile c = walk.at(mt);
            rows = c.rows - 128 * block;
            if (rows <= 0) continue;
            ld = args.ld_sfa;
            src = args.sfa + int64_t(c.row0 + 128 * block) * ld;
            dst = args.atoms_a + (int64_t(c.mt) * KB * 2 + block) * (2 * MM_SF_ATOM / 4);
            step = 2 * (2 * MM_SF_ATOM / 4);
        }
        for (int w0 = 0; w0 < 2 * KB; w0 += 32) {          // 32 words (128 scales) of each row at a time
            const int n = 2 * KB - w0 < 32 ? 2 * KB - w0 : 32;
            if (args.sf_bytes == 16) {                     // k % 512 == 0: whole vectors of 4 words
#pragma unroll 4
                for (int i = threadIdx.x; i < 32 * n; i += 256) {
                    const int r = i / (n / 4), w = 4 * (i - r * (n / 4));
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (r < rows) v = *reinterpret_cast<const uint4 *>(src + r * ld + 4 * (w0 + w));
                    words[r][w] = v.x;
                    words[r][w + 1] = v.y;
                    words[r][w + 2] = v.z;
                    words[r][w + 3] = v.w;
                }
            } else {
                for (int i = threadIdx.x; i < 128 * n; i += 256) {
                    const int r = i / n, w = i - r * n, b = 4 * (w0 + w);
                    uint32_t v = 0u;
                    if (r < rows) {
                        const uint8_t *p = src + r * ld + b;
                        if (args.sf_bytes == 4) {
                            if (b < blocks) v = *reinterpret_cast<const uint32_t *>(p);
                        } else {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (b + x < blocks) v |= static_cast<uint32_t>(p[x]) << (8 * x);
                        }
                    }
                    words[r][w] = v;
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 128 * n; i += 256) {
                const int w = i >> 7, x = i & 127;         // word x of the atom: row x / 4 + 32 (x % 4)
                dst[int64_t((w0 + w) >> 1) * step + ((w0 + w) & 1) * (MM_SF_ATOM / 4) + x] =
                    words[(x >> 2) + 32 * (x & 3)][w];
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- dw = a^T b
struct MmWgradTile {
    int g, row0, rows;   // the expert, or its part (expert * splits + part), and its rows
    int c0, j0, n;       // dw rows and columns; the instruction's N
};

__device__ __forceinline__ MmWgradTile mm_wgrad_tile(int t, int ct, int jt, int width, const int32_t *off)
{
    MmWgradTile w;
    w.g = t / (ct * jt);
    w.row0 = off[w.g];
    w.rows = off[w.g + 1] - w.row0;
    int i, k;
    mm_panel(t - w.g * (ct * jt), ct, jt, i, k);
    w.c0 = i * MM_M;
    w.j0 = k * 256;
    const int left = (width - w.j0 + 15) & ~15;
    w.n = left < 256 ? left : 256;
    return w;
}

// Tensor maps of a and b: 128 bytes (64 elements) x 64 rows.  Both tiles are MN-major (an
// operand's row holds the tile's M or N values at one position of the sum): each CTA has two
// boxes of either a stage (one of double size, as for w above, was no faster here).  The last stage of a group also holds rows of the next one:
// the instructions stop at the next multiple of 16 rows, and the last warp clears the
// rows between, in both operands (what they hold may be NaN, so one is not enough).
template <int GROUPS, typename O, bool LONG>
__global__ void __launch_bounds__(MmWgradCfg<GROUPS>::THREADS, 1)
    mm_wgrad_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_out, const MmArgs args)
{
    using Cfg = MmWgradCfg<GROUPS>;
    constexpr int S = Cfg::STAGES;
    constexpr int KE = 64;   // rows per stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *smem_a = smem;
    uint8_t *smem_b = smem + S * MM_A_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_CTRL);
    uint64_t *full = bars;            // leader: both CTAs' operands landed (and were cleared past the end)
    uint64_t *empty = bars + S;       // both
    uint64_t *tail = bars + 2 * S;    // both: this CTA's copies of a stage that needs clearing landed
    uint64_t *tfull = bars + 3 * S;   // both
    uint64_t *tempty = tfull + 2;     // leader
    uint64_t *drain = tempty + 2;     // leader
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + Cfg::NUM_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile int *begun = abort_flag + 1;   // the tile that this CTA's producer is at
    int32_t *first = reinterpret_cast<int32_t *>(smem + Cfg::OFF_TABLE);
    int32_t *cum = first + (MM_MAX_E + 1);
    // the first row of each expert, or of each part of one: parts are groups like any other
    const int32_t *off = sizeof(O) == 4 && args.splits > 1 ? cum : first;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(&full[s], 2);   // one arrival from each CTA: its producer's, or its clearing warp's
            ptx::mbar_init(&empty[s], 1);
            ptx::mbar_init(&tail[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&tfull[b], 1);
            ptx::mbar_init(&tempty[b], 2 * Cfg::EPI_WARPS);
        }
        ptx::mbar_init(drain, 1);
        *abort_flag = 0;
        *begun = -1;
        ptx::fence_mbar_init();
    }
    if (warp == 0) {
        ptx::pdl_wait_primary();   // what earlier kernels wrote is there for the whole block from the sync below on
        const uint32_t flags = decode_groups_warp(
            args.group_list, args.e, args.group_list_type, args.m, [](int64_t) { return 0; }, first, cum);
        if (off == cum) {
            __syncwarp();
            for (int v = lane; v <= args.e * args.splits; v += 32) {
                const int g = v / args.splits, rows = g < args.e ? first[g + 1] - first[g] : 0;
                // whole stages each but the last
                const int from = (v - g * args.splits) * (((rows + args.splits - 1) / args.splits + 63) & ~63);
                cum[v] = first[g] + (from < rows ? from : rows);
            }
        }
        if (lane == 0) {
            if (blockIdx.x == 0) {
                *args.status = flags;
                for (int g = 0; off == cum && g < args.e; ++g)   // rows, for mm_join_wgrad_kernel
                    args.status[1 + g] = static_cast<uint32_t>(first[g + 1] - first[g]);
            }
            ptx::prefetch_tmap(&map_a);
            ptx::prefetch_tmap(&map_b);
            ptx::prefetch_tmap(&map_out);
        }
    } else if (warp == 1) {
        ptx::tmem_alloc_pair(tmem_holder, 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    ptx::pdl_launch_dependents();
    const uint32_t tmem_base = *tmem_holder;

    const int ct = (args.c + MM_M - 1) / MM_M, jt = (args.j + 255) / 256;
    const int T = args.e * (sizeof(O) == 4 ? args.splits : 1) * ct * jt;
    const int nclusters = mm_active_pairs(T, gridDim.x >> 1);
    const int cluster = static_cast<int>(blockIdx.x >> 1) < nclusters ? blockIdx.x >> 1 : T;   // first tile, or none
    auto tile_at = [&](int t) { return mm_wgrad_tile(t, ct, jt, args.j, off); };

    const uint32_t full_leader0 = ptx::map_to_rank(&full[0], 0);

    auto fail = [&]() {
        atomicOr(args.status, QGMM_DEV_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp == 0) {
        // ------------------------------------------------ copies (both CTAs, own halves)
        if (ptx::elect_one()) {
            constexpr uint32_t HALF = MM_A_BYTES + MM_B_BYTES;
            uint32_t issued = 0;                 // stages handed out
            uint32_t tails = 0, tail_parity = 0; // by stage: its tail barrier was used, and the parity of the last use
            int stage = 0;
            uint32_t phase = 0;
            bool ok = args.stall_producer == 0;
            for (int t = cluster; t < T && ok; t += nclusters) {
                const MmWgradTile c = tile_at(t);
                *begun = t;
                const int c0 = c.c0 + 128 * static_cast<int>(rank);
                const int j0 = c.j0 + c.n / 2 * static_cast<int>(rank);
                for (int r = 0; r < c.rows; r += KE) {
                    if (!ptx::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
                        fail();
                        ok = false;
                        break;
                    }
                    uint8_t *da = smem_a + stage * MM_A_BYTES, *db = smem_b + stage * MM_B_BYTES;
                    const int row = c.row0 + r, left = c.rows - r;
                    const bool clear = left < KE && (left & 15);
                    if (clear) {
                        tail_parity = tails >> stage & 1u ? tail_parity ^ 1u << stage : tail_parity;
                        tails |= 1u << stage;
                        // rows to clear: this CTA's own barrier, then its last warp hands the stage on
                        ptx::mbar_arrive_expect_tx(&tail[stage], HALF);
                        for (int u = 0; u < 2; ++u) {
                            ptx::tma_load_2d(da + u * (MM_A_BYTES / 2), &map_a, &tail[stage], c0 + 64 * u, row);
                            ptx::tma_load_2d(db + u * (MM_B_BYTES / 2), &map_b, &tail[stage], j0 + 64 * u, row);
                        }
                    } else {
                        const uint32_t fb = full_leader0 + stage * 8u;
                        if (leader) ptx::mbar_arrive_expect_tx(&full[stage], 2u * HALF);
                        else ptx::mbar_arrive_cluster(fb);
                        for (int u = 0; u < 2; ++u) {
                            ptx::tma_load_2d_pair(da + u * (MM_A_BYTES / 2), &map_a, fb, c0 + 64 * u, row);
                            ptx::tma_load_2d_pair(db + u * (MM_B_BYTES / 2), &map_b, fb, j0 + 64 * u, row);
                        }
                    }
                    ++issued;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                // let the copies already in flight land before the CTA leaves
                for (uint32_t s = 0; s < S; ++s) {
                    volatile int never = 0;
                    if (tails >> s & 1u) ptx::mbar_wait(&tail[s], tail_parity >> s & 1u, &never);
                    if (issued > s && leader) ptx::mbar_wait(&full[s], ((issued - 1u - s) / S) & 1u, &never);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issue (leader CTA only; as in mm_rows_kernel)
        if (leader && ptx::elect_one()) {
            const uint64_t a_base = ptx::smem_desc_sw128(ptx::smem_addr(smem_a), MM_A_BYTES / 2, 1024);
            const uint64_t b_base = ptx::smem_desc_sw128(ptx::smem_addr(smem_b), MM_B_BYTES / 2, 1024);
            int stage = 0;
            uint32_t phase = 0;
            int lt = 0;
            bool ok = true;
            for (int t = cluster; t < T && ok; t += nclusters) {
                const MmWgradTile c = tile_at(t);
                if (c.rows == 0) continue;
                const uint32_t idesc = ptx::idesc_f16(MM_M, c.n, args.bf16, true, true);
                int buf = 0;
                uint32_t d_tmem = 0;
                bool ready = false;
                for (int r = 0; r < c.rows; r += KE) {
                    const bool first = r / KE % MM_WGRAD_SEGMENT<O, LONG> == 0;
                    const bool last = c.rows - r <= KE || (r / KE + 1) % MM_WGRAD_SEGMENT<O, LONG> == 0;
                    if (first) {
                        buf = lt & 1;
                        const uint32_t use = static_cast<uint32_t>(lt >> 1) & 1u;
                        ++lt;
                        if (!ptx::mbar_wait(&tempty[buf], use ^ 1u, abort_flag)) {
                            fail();
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        d_tmem = tmem_base + static_cast<uint32_t>(buf * 256);
                        ready = ptx::mbar_test_wait_cluster(ptx::smem_addr(&full[stage]), phase);
                    }
                    if (!ready && !ptx::mbar_wait<true>(&full[stage], phase, abort_flag)) {
                        fail();
                        ok = false;
                        break;
                    }
                    const int next = stage + 1 == S ? 0 : stage + 1;
                    const uint32_t next_phase = next ? phase : phase ^ 1u;
                    ready = ptx::mbar_test_wait_cluster(ptx::smem_addr(&full[next]), next_phase);
                    const uint64_t a0 = a_base + stage * (MM_A_BYTES / 16), b0 = b_base + stage * (MM_B_BYTES / 16);
                    const int left = c.rows - r;
#pragma unroll
                    for (int kk = 0; kk < KE / 16; ++kk)
                        if (left > 16 * kk)
                            ptx::mma_f16_pair(d_tmem, a0 + kk * (2048 / 16), b0 + kk * (2048 / 16), idesc,
                                              kk ? 1u : !first);
                    ptx::mma_commit_pair_both(&empty[stage]);
                    if (last) ptx::mma_commit_pair_both(&tfull[buf]);
                    stage = next;
                    phase = next_phase;
                }
            }
            ptx::mma_commit_pair(ptx::map_to_rank(drain, 0));
            volatile int never = 0;
            ptx::mbar_wait(drain, 0, &never);
        }
        __syncwarp();
    } else if (warp < 2 + Cfg::EPI_WARPS) {
        // ------------------------------------------------ epilogue (both CTAs, own 128 dw rows)
        // A thread has one dw row; 128 bytes of 32 rows go through shared memory (16-byte
        // pieces in the 128-byte swizzle, free of conflicts) and leave as one tile copy, which
        // also drops what lies outside dw.  Added to dw, an f32 tile leaves as a reducing copy;
        // 16 bits are added in registers, so that the sum is rounded once.
        const int q = warp & 3, group = (warp - 2) / MM_EPI_WARPS;   // every second chunk of columns
        uint32_t tempty_leader[2];
        tempty_leader[0] = ptx::map_to_rank(&tempty[0], 0);
        tempty_leader[1] = ptx::map_to_rank(&tempty[1], 0);
        uint8_t *stage_mem = smem + Cfg::OFF_STAGING + (warp - 2) * 32 * 128;
        constexpr int W = 128 / sizeof(O);      // columns per chunk
        constexpr int V = 16 / sizeof(O);       // columns per 16-byte piece
        int lt = 0;
        bool ok = true;
        for (int t = cluster; t < T && ok; t += nclusters) {
            const MmWgradTile c = tile_at(t);
            const bool empty_group = c.rows == 0;
            if (empty_group && args.accumulate) continue;
            const int row0 = c.c0 + 128 * static_cast<int>(rank) + 32 * q;
            const int width = args.j - c.j0 < 256 ? args.j - c.j0 : 256;
            O *base = static_cast<O *>(args.out) + static_cast<int64_t>(c.g) * args.out_group +
                      static_cast<int64_t>(row0) * args.ldo + c.j0;
            if (empty_group) {
                for (int w0 = W * group; w0 < width; w0 += W * GROUPS)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = i * 4 + (lane >> 3), p = lane & 7;
                        if (row0 + r < args.c && w0 + p * V < width)
                            *reinterpret_cast<uint4 *>(base + static_cast<int64_t>(r) * args.ldo + w0 + p * V) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                continue;
            }
            constexpr bool IN_REGISTERS = sizeof(O) == 4;
            constexpr int PARTS = 256 / (32 * GROUPS);   // f32: parts of 32 columns of a group
            // 16 bits: this thread's sums of earlier segments, column by column
            float *const kept = args.kept + static_cast<int64_t>(blockIdx.x) * (128 * 256) + 32 * q + lane;
            float sum[IN_REGISTERS ? PARTS : 1][32];
            uint32_t acc = 0;
            const int blocks = (c.rows + KE - 1) / KE;
            int buf = 0;
            for (int block = 0; block < blocks; block += MM_WGRAD_SEGMENT<O, LONG>, ++lt) {
                buf = lt & 1;
                const uint32_t use = static_cast<uint32_t>(lt >> 1) & 1u;
                if (!ptx::mbar_wait_warp(&tfull[buf], use, abort_flag)) {
                    fail();
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                acc = tmem_base + static_cast<uint32_t>(buf * 256) + (static_cast<uint32_t>(32 * q) << 16);
                if constexpr (IN_REGISTERS) {
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        const int w0 = 32 * (group + GROUPS * i);
                        if (w0 >= width) break;
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            uint32_t v[16];
                            ptx::tmem_ld_32x32b_x16(acc + w0 + h, v);
                            ptx::tmem_ld_wait(v);
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                sum[i][h + r] = (block ? sum[i][h + r] : 0.f) + __uint_as_float(v[r]);
                        }
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(tempty_leader[buf]);
                } else if (LONG && blocks - block > MM_WGRAD_SEGMENT<O, LONG>) {
                    for (int w0 = W * group; w0 < width; w0 += W * GROUPS)
                        for (int w = w0; w < w0 + W; w += 16) {
                            float before[16];
#pragma unroll
                            for (int r = 0; r < 16; ++r) before[r] = block ? kept[(w + r) * 128] : 0.f;
                            uint32_t v[16];
                            ptx::tmem_ld_32x32b_x16(acc + w, v);
                            ptx::tmem_ld_wait(v);
#pragma unroll
                            for (int r = 0; r < 16; ++r) kept[(w + r) * 128] = before[r] + __uint_as_float(v[r]);
                        }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(tempty_leader[buf]);
                }
            }
            if (!ok) break;
            auto put = [&](auto more) {
#pragma unroll
                for (int i = 0; i < 256 / (W * GROUPS); ++i) {
                    const int w0 = W * (group + GROUPS * i);
                    if (w0 >= width) break;
                    if (lane == 0) ptx::bulk_wait_read<0>();   // the last copy out of the staging is through
                    __syncwarp();
                    uint4 *dst = reinterpret_cast<uint4 *>(stage_mem + lane * 128);
                    if constexpr (IN_REGISTERS) {
#pragma unroll
                        for (int p = 0; p < 8; ++p)
                            reinterpret_cast<float4 *>(dst)[p ^ (lane & 7)] =
                                make_float4(sum[i][4 * p], sum[i][4 * p + 1], sum[i][4 * p + 2], sum[i][4 * p + 3]);
                    } else {
#pragma unroll
                        for (int h = 0; h < W / 32; ++h) {
                            uint32_t v[32];
                            ptx::tmem_ld_32x32b_x32(acc + w0 + 32 * h, v);
                            ptx::tmem_ld_wait(v);
                            if constexpr (decltype(more)::value) {
#pragma unroll
                                for (int r = 0; r < 32; ++r)
                                    v[r] = __float_as_uint(kept[(w0 + 32 * h + r) * 128] + __uint_as_float(v[r]));
                            }
                            if (!args.accumulate) {
#pragma unroll
                                for (int p = 0; p < 4; ++p) {
                                    uint32_t x[4];
#pragma unroll
                                    for (int u = 0; u < 4; ++u)
                                        x[u] = mm_pack2(static_cast<O *>(nullptr), __uint_as_float(v[8 * p + 2 * u]),
                                                        __uint_as_float(v[8 * p + 2 * u + 1]));
                                    dst[(4 * h + p) ^ (lane & 7)] = make_uint4(x[0], x[1], x[2], x[3]);
                                }
                            } else if (row0 + lane < args.c) {
                                // the sum with what dw holds is rounded once: this thread's own row, in place
                                O *mine = base + static_cast<int64_t>(lane) * args.ldo + w0 + 32 * h;
#pragma unroll
                                for (int p = 0; p < 4; ++p) {
                                    if (w0 + 32 * h + 8 * p >= width) break;
                                    uint4 *at = reinterpret_cast<uint4 *>(mine + 8 * p);
                                    const uint4 o = *at;
                                    const uint32_t old[4] = {o.x, o.y, o.z, o.w};
                                    uint32_t x[4];
#pragma unroll
                                    for (int u = 0; u < 4; ++u) {
                                        const float2 f = mm_unpack2(static_cast<O *>(nullptr), old[u]);
                                        x[u] = mm_pack2(static_cast<O *>(nullptr), f.x + __uint_as_float(v[8 * p + 2 * u]),
                                                        f.y + __uint_as_float(v[8 * p + 2 * u + 1]));
                                    }
                                    *at = make_uint4(x[0], x[1], x[2], x[3]);
                                }
                            }
                            __syncwarp();
                        }
                        if (args.accumulate) continue;
                    }
                    ptx::fence_async_shared();
                    __syncwarp();
                    if (lane == 0 && row0 < args.c) {
                        if (args.accumulate) ptx::tma_reduce_add_3d(&map_out, stage_mem, c.j0 + w0, row0, c.g);
                        else ptx::tma_store_3d(&map_out, stage_mem, c.j0 + w0, row0, c.g);
                        ptx::bulk_commit();
                    }
                }
            };
            if constexpr (LONG) {
                if (blocks > MM_WGRAD_SEGMENT<O, LONG>) put(std::true_type{});
                else put(std::false_type{});
            } else {
                put(std::false_type{});
            }
            if constexpr (!IN_REGISTERS) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(tempty_leader[buf]);
            }
        }
        if (lane == 0) ptx::bulk_wait_all();
        __syncwarp();
    } else {
        // ------------------------------------------------ rows past a group's end (both CTAs)
        int stage = 0;
        uint32_t phase[S];
#pragma unroll
        for (int s = 0; s < S; ++s) phase[s] = 0;
        bool ok = true;
        for (int t = cluster; t < T && ok; t += nclusters) {
            const MmWgradTile c = tile_at(t);
            if (c.rows == 0) continue;
            const int blocks = (c.rows + KE - 1) / KE;
            const int last = (stage + blocks - 1) % S;
            stage = (last + 1) % S;
            const int left = c.rows - (blocks - 1) * KE;
            if (left == KE || !(left & 15)) continue;
            uint32_t parity = 0;
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (s == last) {
                    parity = phase[s];
                    phase[s] ^= 1u;
                }
            // This warp passes the tiles that need no clearing, so it comes here while they are still being
            // summed: its second starts anew while the copies come to further tiles.  (A tile of 2^24 rows
            // takes 0.2 s, at 64 KB a pair and stage from memory.)
            bool landed = false;
            for (bool more = true; more && !landed;) {
                const int before = *begun;
                landed = ptx::mbar_wait_warp(&tail[last], parity, abort_flag);
                more = __any_sync(0xffffffffu, *abort_flag == 0 && *begun != before) != 0;
            }
            if (!landed) {
                fail();
                ok = false;
                break;
            }
            const int clear = 16 - (left & 15);           // rows left .. next multiple of 16
            for (int i = lane; i < clear * 32; i += 32) { // 4 half tiles x 8 pieces of 16 bytes a row
                const int row = left + (i >> 5), atom = (i >> 3) & 3, p = i & 7;
                uint8_t *tile = (atom < 2 ? smem_a : smem_b) + last * MM_A_BYTES + (atom & 1) * (MM_A_BYTES / 2);
                *reinterpret_cast<uint4 *>(tile + row * 128 + p * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            ptx::fence_async_shared();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster_release_smem(full_leader0 + last * 8u);
        }
    }

    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, 512);
    }
}

// Four columns of a call's parts, split_out apart, added up in their order.
__device__ __forceinline__ float4 mm_join4(const float *p, int splits, int64_t split_out)
{
    float4 sum = *reinterpret_cast<const float4 *>(p);
    for (int s = 1; s < splits; ++s) {
        const float4 v = *reinterpret_cast<const float4 *>(p + s * split_out);
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    return sum;
}

__device__ __forceinline__ void mm_store4(float *to, const float4 &v) { *reinterpret_cast<float4 *>(to) = v; }

template <typename O>
__device__ __forceinline__ void mm_store4(O *to, const float4 &v)
{
    *reinterpret_cast<uint2 *>(to) =
        make_uint2(mm_pack2(static_cast<O *>(nullptr), v.x, v.y), mm_pack2(static_cast<O *>(nullptr), v.z, v.w));
}

// out[i][j] = sum_s part[s][i][j] of mm_rows_kernel's parts, rounded once, for the rows that
// the groups cover.
template <typename O>
__global__ void __launch_bounds__(256) mm_join_kernel(const float *part, int splits, int64_t split_out, int j,
                                                      const uint32_t *status, O *out, int64_t ldo)
{
    ptx::pdl_wait_primary();
    ptx::pdl_launch_dependents();
    const int per_row = j / 4;
    const int64_t n = int64_t(status[1]) * per_row;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / per_row;
        const int c = static_cast<int>(i - row * per_row) * 4;
        mm_store4(out + row * ldo + c, mm_join4(part + row * j + c, splits, split_out));
    }
}

// dw[g][i][j] = sum_s part[g][s][i][j] of mm_wgrad_kernel's parts, added to what dw holds with
// `accumulate` (an expert without rows keeps its dw as it is), rounded once.
template <typename O>
__global__ void __launch_bounds__(256) mm_join_wgrad_kernel(const float *part, int splits, int e, int c, int j,
                                                            const uint32_t *status, int accumulate, O *out, int64_t ldo)
{
    ptx::pdl_wait_primary();
    ptx::pdl_launch_dependents();
    const int per_row = j / 4;
    const int64_t split_out = int64_t(c) * j, n = int64_t(e) * c * per_row;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / per_row;     // of e * c
        const int col = static_cast<int>(i - row * per_row) * 4, g = static_cast<int>(row / c);
        if (accumulate && status[1 + g] == 0) continue;
        float4 sum = mm_join4(part + g * splits * split_out + (row - int64_t(g) * c) * j + col, splits, split_out);
        O *to = out + row * ldo + col;
        if (accumulate) {
            float2 lo, hi;
            if constexpr (sizeof(O) == 4) {
                lo = *reinterpret_cast<const float2 *>(to);
                hi = *reinterpret_cast<const float2 *>(to + 2);
            } else {
                const uint2 old = *reinterpret_cast<const uint2 *>(to);
                lo = mm_unpack2(static_cast<O *>(nullptr), old.x);
                hi = mm_unpack2(static_cast<O *>(nullptr), old.y);
            }
            sum = make_float4(lo.x + sum.x, lo.y + sum.y, hi.x + sum.z, hi.y + sum.w);
        }
        mm_store4(to, sum);
    }
}

// The status word of a call that has no rows.
__global__ void mm_status_kernel(const int64_t *group_list, int e, int type, int64_t m, uint32_t *status)
{
    __shared__ int32_t off[MM_MAX_E + 1], cum[MM_MAX_E + 1];
    const uint32_t flags = decode_groups_warp(group_list, e, type, m, [](int64_t) { return 0; }, off, cum);
    if (threadIdx.x == 0) *status = flags;
}

}  // namespace qgmm
