// grouped_mm.cu -- grouped products in bf16, fp16 and MXFP4 and the gradients of the
// 16-bit ones: argument checks, plans and launches for the C ABI in qgmm_mm.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "../../include/qgmm_mm.h"
#include "grouped_mm.cuh"

#define QGMM_MM_API extern "C" __attribute__((visibility("default")))

namespace qgmm {
namespace {

constexpr size_t kWsAlign = 256;
constexpr int64_t kMaxM = int64_t(1) << 24;
constexpr int64_t MM_PLAN_PAIRS = 74;     // pairs of SMs that the splitting and keeping of sums plans for
constexpr int64_t MM_SPLIT_MOST = 32;     // parts
constexpr int64_t MM_SPLIT_SAVES = 24;    // stages that it has to save (MXFP4 and wgrad: half as many)
constexpr int64_t MM_LOW_ROWS = 24;      // rows per expert up to which tiles are low
constexpr int64_t MM_WGRAD_ROWS = 320;   // rows per expert below which the weight gradient takes two epilogue groups
constexpr int64_t MM_ATOMS_ROWS = 384;   // rows per expert from which MXFP4 scales are arranged first

bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int64_t ld_or(int64_t ld, int64_t dense) { return ld ? ld : dense; }

qgmm_status check_problem(const qgmm_mm_problem *p)
{
    if (!p) return QGMM_ERR_NULL_PTR;
    const bool mx = p->x_type == QGMM_T_MXFP4;
    if (p->x_type != QGMM_T_BF16 && p->x_type != QGMM_T_F16 && !mx) return QGMM_ERR_DTYPE;
    if (p->out_type != QGMM_T_F32 && p->out_type != p->x_type &&
        !(mx && (p->out_type == QGMM_T_BF16 || p->out_type == QGMM_T_F16)))
        return QGMM_ERR_DTYPE;
    if (mx && p->out_type == QGMM_T_MXFP4) return QGMM_ERR_DTYPE;
    if (p->group_list_type != QGMM_GROUP_CUMSUM && p->group_list_type != QGMM_GROUP_COUNTS) return QGMM_ERR_DTYPE;
    const int64_t step = mx ? 32 : 8;
    if (p->m < 0 || p->m > kMaxM) return QGMM_ERR_SHAPE;
    if (p->k < step || p->k > 65536 || p->k % step) return QGMM_ERR_SHAPE;
    if (p->n < 8 || p->n > 65536 || p->n % 8) return QGMM_ERR_SHAPE;
    if (p->e < 1 || p->e > MM_MAX_E) return QGMM_ERR_SHAPE;
    if (p->transpose_w != 0 && p->transpose_w != 1) return QGMM_ERR_SHAPE;
    if (p->accumulate != 0 && p->accumulate != 1) return QGMM_ERR_SHAPE;
    if (mx && !p->transpose_w) return QGMM_ERR_UNSUPPORTED;
    if (p->ld_x && (p->ld_x < p->k || p->ld_x % step || p->ld_x > (int64_t(1) << 32))) return QGMM_ERR_SHAPE;
    if (p->ld_w && (p->ld_w < (p->transpose_w ? p->k : p->n) || p->ld_w % step || p->ld_w > (int64_t(1) << 22)))
        return QGMM_ERR_SHAPE;
    if (p->ld_y && (p->ld_y < p->n || p->ld_y % 8 || p->ld_y > (int64_t(1) << 32))) return QGMM_ERR_SHAPE;
    return QGMM_OK;
}

// The workspace: the status word and the count of rows, then for MXFP4 calls with many rows the
// scale words that mm_sf_atoms_kernel arranges, then for few tiles with long sums their parts.
//
// Which calls: the arranging pass reads and writes the scales of every expert with rows
// once, the gathering in the kernel itself costs each row tile a share of its time, so the
// pass pays from about MM_ATOMS_ROWS rows an expert on (k = 2048, n = 7168, 32 experts, quantiser
// included: 256 rows each 102 us with it and 98 without, 1024 rows each 313 and 395).  It also takes the rows
// of scales that no 4-byte load fits (k or a stride not a multiple of 128), which the
// kernel would gather byte by byte.
// The widest load that fits every row of scales: their strides and length k / 32.
int sf_bytes(const qgmm_mm_problem *p)
{
    const int64_t all = (p->k | ld_or(p->ld_x, p->k) | ld_or(p->ld_w, p->k)) / 32;
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
}

// Greatest height of a row tile.  A call that cannot have a higher one, or whose experts have
// MM_LOW_ROWS rows or fewer on average, takes low tiles and the longer ring that goes with
// them (8 rows over 8 experts 43.3 us against 45.7, 256 to 768 rows over 32 experts within 2%).
int tile_height(const qgmm_mm_problem *p)
{
    const int64_t groups = p->e < p->m ? p->e : p->m;
    if (p->m <= MM_LOW_N || p->m <= MM_LOW_ROWS * groups) return MM_LOW_N;
    return p->x_type == QGMM_T_MXFP4 ? MmRowsCfg<MM_MXF4>::TILE_N : MmRowsCfg<MM_F16>::TILE_N;
}

struct MmAtoms {
    bool use;
    int64_t units_w, units_a;   // KB of scale words: w's, and the row tiles'
    size_t w, a, total;
};

MmAtoms mm_atoms(const qgmm_mm_problem *p)
{
    MmAtoms A = {};
    A.total = kWsAlign;
    A.use = p->x_type == QGMM_T_MXFP4 && (p->m >= MM_ATOMS_ROWS * p->e || sf_bytes(p) == 1);
    if (!A.use) return A;
    const int64_t height = tile_height(p), groups = p->e < p->m ? p->e : p->m;
    const int64_t kb = (p->k + 255) / 256, tiles = (p->m + height - 1) / height + groups;
    A.units_w = p->e * 2 * ((p->n + MM_M - 1) / MM_M) * kb;
    A.units_a = tiles * kb * 2;
    A.w = kWsAlign;
    A.a = A.w + size_t(A.units_w) * 1024;
    A.total = A.a + size_t(A.units_a) * 1024;
    return A;
}

// The parts of a sum.  Tiles that are fewer than half the pairs leave pairs idle, and a pair
// alone walks a long sum at the latency of its copies (0.2 us a stage of bf16, 0.4 us of MXFP4);
// then each tile's sum is cut into parts of split_kb stages for as many pairs, whose f32
// results the workspace holds until mm_join_kernel adds them up in order.  That launch costs
// 3 to 4 us, and every 2^18 f32 of the parts about as much as a stage, so the parts have to save
// more stages than that.  (One row, bf16, us whole and in parts: k = 4096 n = 1024 16.5 and 11.5,
// k = 8192 28.6 and 13.5, k = 65536 n = 256 194 and 19.2, but k = 2048 n = 1024 10.6 and 11.4;
// MXFP4 k = 16384 n = 256 22.3 and 10.4.  2048 rows, n = 512: k = 4096 26.0 and 23.9,
// k = 2048 16.5 and 20.7.  8 parts at most: k = 65536 34.3.)
struct MmSplit {
    int splits, split_kb;
    size_t at, total;      // byte offset of the parts (or of kept sums), and the workspace with them
};

MmSplit mm_split(const qgmm_mm_problem *p, bool dgrad)
{
    MmSplit S = {1, 0, 0, mm_atoms(p).total};
    const int64_t c = dgrad ? p->n : p->k, j = dgrad ? p->k : p->n, height = tile_height(p);
    const int64_t kb = (c + (p->x_type == QGMM_T_MXFP4 ? 255 : 63)) / (p->x_type == QGMM_T_MXFP4 ? 256 : 64);
    const int64_t groups = p->e < p->m ? p->e : p->m;
    const int64_t tiles = ((p->m - groups) / height + groups) * ((j + MM_M - 1) / MM_M);   // at most
    if (p->m == 0 || 2 * tiles > MM_PLAN_PAIRS) return S;
    const int64_t most = MM_PLAN_PAIRS / tiles < MM_SPLIT_MOST ? MM_PLAN_PAIRS / tiles : MM_SPLIT_MOST;
    const int64_t part = ((kb + most - 1) / most + 7) / 8 * 8;   // whole segments, and pieces of scales
    const int64_t splits = (kb + part - 1) / part;
    const int64_t cost = MM_SPLIT_SAVES / (p->x_type == QGMM_T_MXFP4 ? 2 : 1) + (splits * p->m * j >> 18);
    if (kb - part <= cost) return S;
    S.split_kb = static_cast<int>(part);
    S.splits = static_cast<int>(splits);
    S.at = S.total;
    S.total = S.at + size_t(S.splits) * size_t(p->m) * size_t(j) * 4;
    S.total = (S.total + kWsAlign - 1) / kWsAlign * kWsAlign;
    return S;
}

// Bytes of the sums that a weight gradient keeps between segments: none unless an expert may have rows for two.
size_t kept_bytes(const qgmm_mm_problem *p)
{
    if (p->out_type == QGMM_T_F32) return 0;
    const int64_t stages = p->out_type == QGMM_T_BF16 ? MM_LONG_SEGMENT<__nv_bfloat16> : MM_LONG_SEGMENT<__half>;
    const int64_t tiles = p->e * ((p->k + 255) / 256) * ((p->n + 255) / 256);
    return p->m <= 64 * stages ? 0 : size_t(MM_KEPT_BYTES) * size_t(tiles < MM_PLAN_PAIRS ? tiles : MM_PLAN_PAIRS);
}

// The same for the weight gradient, whose sum runs over an expert's rows: the parts' lengths follow
// from the groups on the device, their number from the rows that an expert has on average.
// (fp16 to f32, us whole and in parts: one expert, 65536 rows, k = n = 256 303 and 26.7, 2048 rows,
// k = 64 n = 256 15.8 and 11.2, 4096 rows, k = 2048 n = 1024 28.2 and 25.5; 13877 rows of three
// experts, k = 152 n = 72 54.3 and 13.8.)
// Whole sums of 16-bit outputs with more than one segment are kept there between them, a tile for each pair.
MmSplit mm_split_wgrad(const qgmm_mm_problem *p)
{
    const size_t at = mm_atoms(p).total;
    MmSplit S = {1, 0, at, at};
    const int64_t kb = (p->m / p->e + 63) / 64;
    const int64_t tiles = p->e * ((p->k + 255) / 256) * ((p->n + 255) / 256);
    S.total += kept_bytes(p);
    if (p->m == 0 || 2 * tiles > MM_PLAN_PAIRS) return S;
    int64_t splits = MM_PLAN_PAIRS / tiles < MM_SPLIT_MOST ? MM_PLAN_PAIRS / tiles : MM_SPLIT_MOST;
    if (splits > kb / 8) splits = kb / 8;
    if (splits < 2 || kb - kb / splits <= MM_SPLIT_SAVES / 2 + (splits * p->e * p->k * p->n >> 18)) return S;
    S.splits = static_cast<int>(splits);
    S.total = S.at + size_t(splits) * size_t(p->e) * size_t(p->k) * size_t(p->n) * 4;
    S.total = (S.total + kWsAlign - 1) / kWsAlign * kWsAlign;
    return S;
}

// Bytes of a call's workspace, any of the three.
size_t workspace_of(const qgmm_mm_problem *p)
{
    size_t most = mm_split(p, false).total;
    if (p->x_type == QGMM_T_MXFP4) return most;   // no gradients
    const size_t back = mm_split(p, true).total, w = mm_split_wgrad(p).total;
    if (most < back) most = back;
    return most < w ? w : most;
}

// The same with p->m rows or fewer, so that the workspace of the largest batch serves every other.
// Calls of few rows are cut into parts, and low tiles take more arranged scales than high ones.
size_t workspace_up_to(const qgmm_mm_problem *p)
{
    size_t most = workspace_of(p);
    qgmm_mm_problem s = *p;
    auto look = [&](int64_t rows) {
        s.m = rows < p->m ? rows : p->m;
        return &s;
    };
    auto take = [&](size_t bytes) { most = most < bytes ? bytes : most; };
    const bool mx = p->x_type == QGMM_T_MXFP4;
    take(workspace_of(look(MM_LOW_ROWS * p->e < MM_LOW_N ? MM_LOW_N : MM_LOW_ROWS * p->e)));   // the last of low tiles
    for (int dgrad = 0; dgrad < (mx ? 1 : 2); ++dgrad) {
        // parts: at most half the pairs have a tile, which is 256 rows at most
        const int64_t cols = ((dgrad ? p->k : p->n) + MM_M - 1) / MM_M, last = MM_PLAN_PAIRS / 2 / cols * 256;
        for (int64_t m = 1; m <= last && m <= p->m; ++m) {
            if ((m < p->e ? m : p->e) * cols > MM_PLAN_PAIRS / 2) break;   // every expert with rows has a tile
            take(mm_split(look(m), dgrad != 0).total);
        }
    }
    if (mx) return most;
    // the weight gradient's: their number grows with the stages of an average expert, up to MM_SPLIT_MOST for 8 each
    for (int64_t kb = 1; kb <= 9 * MM_SPLIT_MOST && 64 * (kb - 1) * p->e < p->m; ++kb)
        take(mm_split_wgrad(look(64 * kb * p->e)).total);
    take(mm_atoms(p).total + kept_bytes(p));
    return most;
}

qgmm_status check_call(const qgmm_mm_problem *p, const void *group_list, const void *workspace, size_t ws_bytes)
{
    if (!group_list || !workspace) return QGMM_ERR_NULL_PTR;
    if (misaligned(workspace, kWsAlign)) return QGMM_ERR_ALIGNMENT;
    return ws_bytes < workspace_of(p) ? QGMM_ERR_WORKSPACE_TOO_SMALL : QGMM_OK;
}

// ---------------------------------------------------------------- tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// `rank`-dimensional map, by default 128-byte rows in the 128-byte swizzle, zeros outside: dim[0] elements
// of `type` contiguous, stride[i] bytes from one index of dim[i + 1] to the next.
qgmm_status make_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dim,
                     const cuuint64_t *stride, uint32_t box_x, uint32_t box_y, bool swizzle = true, uint32_t box_z = 1)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return QGMM_ERR_CUDA;
    const cuuint32_t box[4] = {box_x, box_y, box_z, 1}, es[4] = {1, 1, 1, 1};
    return enc(map, type, rank, const_cast<void *>(base), dim, stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QGMM_OK
               : QGMM_ERR_CUDA;
}

// The maps of a row operand: half the greatest tile's rows, and lower boxes.
qgmm_status make_row_maps(MmRowsMaps *maps, CUtensorMapDataType type, const void *base, const cuuint64_t *dim,
                          const cuuint64_t *stride, uint32_t box_x, uint32_t tall)
{
    qgmm_status s = make_map(&maps->a, type, 2, base, dim, stride, box_x, tall);
    for (int b = 0; b < 4 && s == QGMM_OK; ++b) s = make_map(&maps->low[b], type, 2, base, dim, stride, box_x, 64u >> b);
    return s;
}

// ---------------------------------------------------------------- launches
constexpr int kMaxDevices = 64;
std::mutex g_mu;

// Launch `kern` on pairs: at most `tiles` of them, and no more than fit the device at once.
// Every kernel here may start beside the one before it on the stream, and waits for that one's
// results itself (griddepcontrol): a call's prologue costs nothing behind another call.
template <typename K, typename... Args>
qgmm_status launch_pairs(K kern, int *clusters_of_device, int threads, size_t smem, int64_t tiles, cudaStream_t st,
                         Args... args)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return QGMM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;   // the occupancy query below uses the cluster shape only
    int clusters = 0;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (clusters_of_device[dev] == 0) {   // first call on this device
            int sms = 0, major = 0;
            if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
                return QGMM_ERR_CUDA;
            if (major != 10) return QGMM_ERR_UNSUPPORTED;
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
                return QGMM_ERR_CUDA;
            cfg.gridDim = dim3(static_cast<unsigned>(sms & ~1), 1, 1);
            if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1)
                return QGMM_ERR_CUDA;
            clusters_of_device[dev] = clusters;
        }
        clusters = clusters_of_device[dev];
    }
    const int64_t pairs = tiles < clusters ? (tiles < 1 ? 1 : tiles) : clusters;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
    cfg.numAttrs = 2;
    // (its own answer: cudaGetLastError would also report what an earlier call left behind)
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? QGMM_OK : QGMM_ERR_CUDA;
}

template <int KIND, typename O, bool LONG>
qgmm_status launch_rows_t(const MmRowsMaps &maps, const MmArgs &args, cudaStream_t st)
{
    using Cfg = MmRowsCfg<KIND>;
    static int clusters[kMaxDevices];
    const int64_t groups = args.e < args.m ? args.e : args.m;
    const int64_t tiles = ((args.m + args.tile_n - 1) / args.tile_n + groups) * ((args.j + MM_M - 1) / MM_M) *
                          args.splits;
    return launch_pairs(mm_rows_kernel<KIND, O, LONG>, clusters, Cfg::THREADS, Cfg::SMEM_BYTES, tiles, st, maps, args);
}

template <int KIND, typename O>
qgmm_status launch_rows(const MmRowsMaps &maps, const MmArgs &args, cudaStream_t st)
{
    if constexpr (KIND == MM_F16 && sizeof(O) == 2)
        if (args.c > MM_LONG_TERMS) return launch_rows_t<KIND, O, true>(maps, args, st);
    return launch_rows_t<KIND, O, false>(maps, args, st);
}

template <int GROUPS, typename O, bool LONG>
qgmm_status launch_wgrad_t(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &out, const MmArgs &args,
                           cudaStream_t st)
{
    using Cfg = MmWgradCfg<GROUPS>;
    static int clusters[kMaxDevices];
    int64_t tiles = int64_t(args.e) * args.splits * ((args.c + MM_M - 1) / MM_M) * ((args.j + 255) / 256);
    if (LONG && tiles > MM_PLAN_PAIRS) tiles = MM_PLAN_PAIRS;   // the pairs that the workspace has room for
    return launch_pairs(mm_wgrad_kernel<GROUPS, O, LONG>, clusters, Cfg::THREADS, Cfg::SMEM_BYTES, tiles, st, a, b, out, args);
}

// Two epilogue groups where an expert's rows are few and storing dw is the bound, one (and
// the longer ring) where they are many and the products are: 32 experts, k = 2048, n = 7168,
// bf16, us with two and with one: 128 rows each 198 and 208, 256 rows 276 and 276, 512 rows
// 428 and 415.  f32 sums need the registers of two.
template <typename O>
qgmm_status launch_wgrad(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &out, const MmArgs &args,
                         cudaStream_t st)
{
    if constexpr (sizeof(O) == 2) {
        const bool one = args.m >= MM_WGRAD_ROWS * args.e;
        if (args.kept)
            return one ? launch_wgrad_t<1, O, true>(a, b, out, args, st) : launch_wgrad_t<2, O, true>(a, b, out, args, st);
        if (one) return launch_wgrad_t<1, O, false>(a, b, out, args, st);
    }
    return launch_wgrad_t<2, O, false>(a, b, out, args, st);
}

MmArgs base_args(const qgmm_mm_problem *p, const int64_t *group_list, void *out, void *workspace)
{
    MmArgs a = {};
    a.group_list = group_list;
    a.group_list_type = p->group_list_type;
    a.e = static_cast<int32_t>(p->e);
    a.m = p->m;
    a.bf16 = p->x_type == QGMM_T_BF16;
    a.out = out;
    a.status = static_cast<uint32_t *>(workspace);
    // Test hook of the failure path: no copy is issued, every wait runs out after its second,
    // the kernel sets QGMM_DEV_TIMEOUT, frees its tensor memory and returns.
    const char *stall = std::getenv("QGMM_TEST_STALL_PRODUCER");
    a.stall_producer = stall && std::atoi(stall) != 0;
    a.splits = 1;
    return a;
}

qgmm_status launch_atoms(const MmArgs &a, int64_t units, cudaStream_t st)
{
    // a block arranges `units` KB in turn: enough blocks for every SM to hold eight
    const int grid = static_cast<int>(units < 1184 ? units : 1184);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mm_sf_atoms_kernel, a) == cudaSuccess ? QGMM_OK
                                                                                                      : QGMM_ERR_CUDA;
}

template <typename K, typename... Args>
qgmm_status launch_join_kernel(K kern, int64_t quads, cudaStream_t st, Args... args)
{
    const int64_t blocks = (quads + 255) / 256;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < 1184 ? blocks : 1184), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? QGMM_OK : QGMM_ERR_CUDA;
}

template <typename O>
qgmm_status launch_join_t(const MmArgs &a, void *out, int64_t ldo, cudaStream_t st)
{
    return launch_join_kernel(mm_join_kernel<O>, a.m * (a.j / 4), st, static_cast<const float *>(a.out), int(a.splits),
                              a.split_out, int(a.j), static_cast<const uint32_t *>(a.status), static_cast<O *>(out), ldo);
}

template <typename O>
qgmm_status launch_join_wgrad_t(const MmArgs &a, int accumulate, void *out, int64_t ldo, cudaStream_t st)
{
    return launch_join_kernel(mm_join_wgrad_kernel<O>, int64_t(a.e) * a.c * (a.j / 4), st, static_cast<const float *>(a.out),
                              int(a.splits), int(a.e), int(a.c), int(a.j), static_cast<const uint32_t *>(a.status),
                              accumulate, static_cast<O *>(out), ldo);
}

qgmm_status launch_join(const MmArgs &a, int32_t type, void *out, int64_t ldo, cudaStream_t st)
{
    return type == QGMM_T_F32    ? launch_join_t<float>(a, out, ldo, st)
           : type == QGMM_T_BF16 ? launch_join_t<__nv_bfloat16>(a, out, ldo, st)
                                 : launch_join_t<__half>(a, out, ldo, st);
}

qgmm_status launch_join_wgrad(const MmArgs &a, int32_t type, int accumulate, void *out, int64_t ldo, cudaStream_t st)
{
    return type == QGMM_T_F32    ? launch_join_wgrad_t<float>(a, accumulate, out, ldo, st)
           : type == QGMM_T_BF16 ? launch_join_wgrad_t<__nv_bfloat16>(a, accumulate, out, ldo, st)
                                 : launch_join_wgrad_t<__half>(a, accumulate, out, ldo, st);
}

qgmm_status launch_status(const MmArgs &a, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(32, 1, 1);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, mm_status_kernel, a.group_list, a.e, a.group_list_type, a.m, a.status) == cudaSuccess
               ? QGMM_OK
               : QGMM_ERR_CUDA;
}

qgmm_status rows_product(const qgmm_mm_problem *p, bool dgrad, const void *x, const uint8_t *sfx, const void *w,
                         const uint8_t *sfw, const int64_t *group_list, void *out, void *workspace, size_t ws_bytes,
                         void *cuda_stream)
{
    qgmm_status s = check_problem(p);
    if (s != QGMM_OK) return s;
    const bool mx = p->x_type == QGMM_T_MXFP4;
    if (p->accumulate || (dgrad && mx)) return QGMM_ERR_UNSUPPORTED;
    if ((s = check_call(p, group_list, workspace, ws_bytes)) != QGMM_OK) return s;
    if (!w || (mx && !sfw)) return QGMM_ERR_NULL_PTR;
    if (p->m && (!x || !out || (mx && !sfx))) return QGMM_ERR_NULL_PTR;
    if (misaligned(x, 16) || misaligned(w, 16) || misaligned(out, 16) || misaligned(sfx, 16) || misaligned(sfw, 16))
        return QGMM_ERR_ALIGNMENT;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    MmArgs a = base_args(p, group_list, out, workspace);
    if (p->m == 0) return launch_status(a, st);

    const int64_t ldx = ld_or(p->ld_x, p->k), ldy = ld_or(p->ld_y, p->n);
    const int64_t ldw = ld_or(p->ld_w, p->transpose_w ? p->k : p->n);
    a.c = static_cast<int32_t>(dgrad ? p->n : p->k);
    a.j = static_cast<int32_t>(dgrad ? p->k : p->n);
    const int64_t ldo = dgrad ? ldx : ldy;
    a.ldo = ldo;
    a.w_mn = (p->transpose_w != 0) == dgrad;   // w's rows run along the output's columns
    a.sfa = sfx;
    a.sfw = sfw;
    a.ld_sfa = ldx / 32;
    a.ld_sfw = ldw / 32;
    a.sf_bytes = sf_bytes(p);
    const MmAtoms A = mm_atoms(p);
    a.sf_atoms = A.use;
    a.tile_n = tile_height(p);
    const uint64_t cols = (uint64_t(a.j) + MM_M - 1) / MM_M;
    a.cols_magic = ((uint64_t(1) << 40) + cols - 1) / cols;

    const MmSplit S = mm_split(p, dgrad);
    a.splits = S.splits;
    a.split_kb = S.split_kb;
    if (S.splits > 1) {
        a.out = static_cast<uint8_t *>(workspace) + S.at;
        a.ldo = a.j;
        a.split_out = p->m * a.j;
    }
    const int32_t kernel_type = S.splits > 1 ? QGMM_T_F32 : p->out_type;
    MmRowsMaps maps = {};
    if (kernel_type != QGMM_T_F32) {
        const cuuint64_t od[2] = {cuuint64_t(a.j), cuuint64_t(p->m)}, ost[1] = {cuuint64_t(a.ldo) * 2};
        if ((s = make_map(&maps.out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, out, od, ost, 64, MM_OUT_ROWS)) != QGMM_OK)
            return s;
    }
    const cuuint64_t lda = cuuint64_t(dgrad ? ldy : ldx), c = cuuint64_t(a.c), j = cuuint64_t(a.j);
    const cuuint64_t w_rows = cuuint64_t(p->transpose_w ? p->n : p->k);
    if (mx) {
        const cuuint64_t wd[3] = {c / 2, j, cuuint64_t(p->e)}, wst[2] = {cuuint64_t(ldw) / 2, w_rows * ldw / 2};
        const cuuint64_t ad[2] = {c / 2, cuuint64_t(p->m)}, ast[1] = {lda / 2};
        const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_UINT8;
        if ((s = make_map(&maps.w, t, 3, w, wd, wst, 128, 128)) != QGMM_OK ||
            (s = make_row_maps(&maps, t, x, ad, ast, 128, MmRowsCfg<MM_MXF4>::TILE_N / 2)) != QGMM_OK)
            return s;
        if (A.use) {
            a.atoms_w = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + A.w);
            a.atoms_a = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + A.a);
            const cuuint64_t swd[2] = {256, cuuint64_t(A.units_w)}, sad[2] = {256, cuuint64_t(A.units_a)};
            const cuuint64_t kb[1] = {1024};
            if ((s = make_map(&maps.sfw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, a.atoms_w, swd, kb, 256, 1, false)) != QGMM_OK ||
                (s = make_map(&maps.sfa, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, a.atoms_a, sad, kb, 256, 2, false)) != QGMM_OK ||
                (s = launch_atoms(a, A.units_w + A.units_a, st)) != QGMM_OK)
                return s;
        }
        switch (kernel_type) {
        case QGMM_T_F32: s = launch_rows<MM_MXF4, float>(maps, a, st); break;
        case QGMM_T_BF16: s = launch_rows<MM_MXF4, __nv_bfloat16>(maps, a, st); break;
        default: s = launch_rows<MM_MXF4, __half>(maps, a, st);
        }
        return s == QGMM_OK && S.splits > 1 ? launch_join(a, p->out_type, out, ldo, st) : s;
    }
    const cuuint64_t ad[2] = {c, cuuint64_t(p->m)}, ast[1] = {lda * 2};
    const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_UINT16;
    if (a.w_mn && j % 64 == 0) {
        // (e, c, j) as (e, j / 64, c, 64): two neighbouring blocks of 64 j in one copy
        a.w_blocks = 1;
        const cuuint64_t wd[4] = {64, c, j / 64, cuuint64_t(p->e)};
        const cuuint64_t wst[3] = {cuuint64_t(ldw) * 2, 128, w_rows * ldw * 2};
        s = make_map(&maps.w, t, 4, w, wd, wst, 64, 64, true, 2);
    } else {
        const cuuint64_t wd[3] = {a.w_mn ? j : c, a.w_mn ? c : j, cuuint64_t(p->e)};
        const cuuint64_t wst[2] = {cuuint64_t(ldw) * 2, w_rows * ldw * 2};
        s = make_map(&maps.w, t, 3, w, wd, wst, 64, a.w_mn ? 64 : 128);
    }
    if (s != QGMM_OK || (s = make_row_maps(&maps, t, x, ad, ast, 64, MmRowsCfg<MM_F16>::TILE_N / 2)) != QGMM_OK) return s;
    switch (kernel_type) {
    case QGMM_T_F32: s = launch_rows<MM_F16, float>(maps, a, st); break;
    case QGMM_T_BF16: s = launch_rows<MM_F16, __nv_bfloat16>(maps, a, st); break;
    default: s = launch_rows<MM_F16, __half>(maps, a, st);
    }
    return s == QGMM_OK && S.splits > 1 ? launch_join(a, p->out_type, out, ldo, st) : s;
}

}  // namespace
}  // namespace qgmm

using namespace qgmm;

QGMM_MM_API qgmm_status qgmm_grouped_mm_workspace(const qgmm_mm_problem *p, size_t *ws_bytes)
{
    if (!ws_bytes) return QGMM_ERR_NULL_PTR;
    const qgmm_status s = check_problem(p);
    if (s != QGMM_OK) return s;
    *ws_bytes = workspace_up_to(p);
    return QGMM_OK;
}

QGMM_MM_API qgmm_status qgmm_grouped_mm(const qgmm_mm_problem *p, const void *x, const uint8_t *x_scale, const void *w,
                                        const uint8_t *w_scale, const int64_t *group_list, void *y, void *workspace,
                                        size_t ws_bytes, void *cuda_stream)
{
    return rows_product(p, false, x, x_scale, w, w_scale, group_list, y, workspace, ws_bytes, cuda_stream);
}

QGMM_MM_API qgmm_status qgmm_grouped_mm_dgrad(const qgmm_mm_problem *p, const void *dy, const void *w,
                                              const int64_t *group_list, void *dx, void *workspace, size_t ws_bytes,
                                              void *cuda_stream)
{
    return rows_product(p, true, dy, nullptr, w, nullptr, group_list, dx, workspace, ws_bytes, cuda_stream);
}

QGMM_MM_API qgmm_status qgmm_grouped_mm_wgrad(const qgmm_mm_problem *p, const void *x, const void *dy,
                                              const int64_t *group_list, void *dw, void *workspace, size_t ws_bytes,
                                              void *cuda_stream)
{
    qgmm_status s = check_problem(p);
    if (s != QGMM_OK) return s;
    if (p->x_type == QGMM_T_MXFP4) return QGMM_ERR_UNSUPPORTED;
    if ((s = check_call(p, group_list, workspace, ws_bytes)) != QGMM_OK) return s;
    if (!dw || (p->m && (!x || !dy))) return QGMM_ERR_NULL_PTR;
    if (misaligned(x, 16) || misaligned(dy, 16) || misaligned(dw, 16)) return QGMM_ERR_ALIGNMENT;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    MmArgs a = base_args(p, group_list, dw, workspace);
    // dw's rows are the dimension the M side covers, its columns the N side's
    const bool t = p->transpose_w != 0;
    a.c = static_cast<int32_t>(t ? p->n : p->k);
    a.j = static_cast<int32_t>(t ? p->k : p->n);
    const MmSplit S = mm_split_wgrad(p);
    const int64_t ldo = ld_or(p->ld_w, a.j);
    void *out = dw;
    a.ldo = ldo;
    a.accumulate = p->accumulate;
    if (S.splits > 1) {
        a.splits = S.splits;
        out = a.out = static_cast<uint8_t *>(workspace) + S.at;
        a.ldo = a.j;
        a.accumulate = 0;
    } else if (S.total > S.at) {
        a.kept = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + S.at);
    }
    a.out_group = a.c * a.ldo;
    const int64_t ldx = ld_or(p->ld_x, p->k), ldy = ld_or(p->ld_y, p->n);
    // without rows nothing is copied: the maps then only have to be valid
    const void *pa = p->m ? (t ? dy : x) : dw, *pb = p->m ? (t ? x : dy) : dw;
    const cuuint64_t rows = cuuint64_t(p->m ? p->m : 1);
    const int64_t lda = t ? ldy : ldx, ldb = t ? ldx : ldy;
    const bool f32 = p->out_type == QGMM_T_F32 || S.splits > 1;
    const cuuint64_t size = f32 ? 4 : 2;
    const cuuint64_t od[3] = {cuuint64_t(a.j), cuuint64_t(a.c), cuuint64_t(p->e) * a.splits};
    const cuuint64_t ost[2] = {cuuint64_t(a.ldo) * size, cuuint64_t(a.out_group) * size};
    CUtensorMap mo, mab[2];
    if ((s = make_map(&mo, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, out, od, ost,
                      uint32_t(128 / size), 32)) != QGMM_OK)
        return s;
    for (int o = 0; o < 2; ++o) {
        const cuuint64_t width = cuuint64_t(o ? a.j : a.c), ld = cuuint64_t(o ? ldb : lda) * 2;
        const void *base = o ? pb : pa;
        const cuuint64_t dim[2] = {width, rows}, stride[1] = {ld};
        s = make_map(&mab[o], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, dim, stride, 64, 64);
        if (s != QGMM_OK) return s;
    }
    if (f32) {
        s = launch_wgrad<float>(mab[0], mab[1], mo, a, st);
        return s == QGMM_OK && S.splits > 1 ? launch_join_wgrad(a, p->out_type, p->accumulate, dw, ldo, st) : s;
    }
    return p->x_type == QGMM_T_BF16 ? launch_wgrad<__nv_bfloat16>(mab[0], mab[1], mo, a, st)
                                    : launch_wgrad<__half>(mab[0], mab[1], mo, a, st);
}
