// mxfp4.cu -- MXFP4 quantisation and its inverse: E2M1 values, two per byte, with an
// E8M0 scale per 32 consecutive elements of a row (qgmm_mm.h has the formulas).
//
// Both kernels are one pass over memory.  (Their pointers are not __restrict__: loads that
// the compiler may take for invariant could move above the wait for the kernel before.)  A thread takes 8 elements, four
// neighbouring threads a block of 32: 16-byte loads of 16-bit types, coalesced over
// the warp, two shuffles for the block's maximum, a 4-byte store of codes.  Rows are
// dense and k % 32 == 0, so the tensor is one run of blocks and rows do not matter.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/qgmm_mm.h"
#include "ptx_sm100.cuh"

#define QGMM_MM_API extern "C" __attribute__((visibility("default")))

namespace qgmm {
namespace {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;      // pieces a thread holds at once: quantiser (2 and 8 measured the same or slower)
constexpr int UNROLL_OUT = 8;  // and expansion, whose loads are short (83 us against 88 with 4 at 57344 x 2048)

struct alignas(16) Vec16 { uint32_t w[4]; };

// 8 consecutive elements as f32 (exact).
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8])
{
    const Vec16 h = *reinterpret_cast<const Vec16 *>(p);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        v[2 * u] = __uint_as_float(h.w[u] << 16);
        v[2 * u + 1] = __uint_as_float(h.w[u] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load8(const __half *p, float (&v)[8])
{
    const Vec16 h = *reinterpret_cast<const Vec16 *>(p);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h.w[u]));
        v[2 * u] = f.x;
        v[2 * u + 1] = f.y;
    }
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const float4 f = reinterpret_cast<const float4 *>(p)[u];
        v[4 * u] = f.x;
        v[4 * u + 1] = f.y;
        v[4 * u + 2] = f.z;
        v[4 * u + 3] = f.w;
    }
}

// 16 bytes of the first values, each rounded once to nearest even.
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&v)[8])
{
    Vec16 h;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * u], v[2 * u + 1]);
        h.w[u] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<Vec16 *>(p) = h;
}

__device__ __forceinline__ void store16(__half *p, const float (&v)[8])
{
    Vec16 h;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const __half2 b = __floats2half2_rn(v[2 * u], v[2 * u + 1]);
        h.w[u] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<Vec16 *>(p) = h;
}

__device__ __forceinline__ void store16(float *p, const float (&v)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

template <int W> struct CodesOf { using type = uint32_t; };   // W codes
template <> struct CodesOf<4> { using type = uint16_t; };

// 8 values to 8 E2M1 codes, the first in the lowest nibble (nearest even, 6 at most).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The value of the lowest E2M1 code, exact: its exponent and mantissa bits at the foot of
// f32's exponent give the value times 2^-126 (the subnormal 0.5 included).
__device__ __forceinline__ float e2m1_value(uint32_t code)
{
    return __uint_as_float((code & 8u) << 28 | (code & 7u) << 22) * 0x1p126f;
}

// `eighths` 8-element pieces, a multiple of 4: the four lanes of a block are in or out
// of range together, and so is a whole quad's shuffle.
template <typename T>
__global__ void __launch_bounds__(THREADS) quant_mxfp4_kernel(const T *x, int64_t eighths, uint32_t *q,
                                                              uint8_t *sf)
{
    ptx::pdl_wait_primary();
    ptx::pdl_launch_dependents();
    const int64_t i0 = blockIdx.x * int64_t(THREADS * UNROLL) + threadIdx.x;
    float v[UNROLL][8];
#pragma unroll
    for (int r = 0; r < UNROLL; ++r) {
        const int64_t i = i0 + r * THREADS;
#pragma unroll
        for (int u = 0; u < 8; ++u) v[r][u] = 0.f;
        if (i < eighths) load8(x + i * 8, v[r]);
    }
#pragma unroll
    for (int r = 0; r < UNROLL; ++r) {
        const int64_t i = i0 + r * THREADS;
        // |x| as integers order like the magnitudes, infinity above them and NaN above that
        uint32_t a = 0u;
#pragma unroll
        for (int u = 0; u < 8; ++u) a = max(a, __float_as_uint(v[r][u]) & 0x7FFFFFFFu);
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const bool nan = a > 0x7F800000u;
        const int biased = static_cast<int>(a >> 23);
        const int code = biased > 2 ? biased - 2 : 0;
        const float inv = nan ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - code) << 23);   // 2^(127 - code)
#pragma unroll
        for (int u = 0; u < 8; ++u) v[r][u] = __fmul_rn(v[r][u], inv);
        if (i < eighths) {
            q[i] = nan ? 0u : e2m1x8(v[r]);
            if ((threadIdx.x & 3) == 0) sf[i >> 2] = static_cast<uint8_t>(nan ? 255 : code);
        }
    }
}

// A thread stores 16 bytes at a time, its neighbours the next ones: W = 8 elements of the
// 16-bit types, 4 of f32 (8 a thread would leave every store half a sector apart: 140
// against 80 us at 57344 x 2048).  `pieces` of W elements, each inside one block.
template <typename T>
__global__ void __launch_bounds__(THREADS) dequant_mxfp4_kernel(const uint8_t *q, const uint8_t *sf,
                                                                int64_t pieces, T *out)
{
    constexpr int W = 16 / sizeof(T);
    using Codes = typename CodesOf<W>::type;
    ptx::pdl_wait_primary();
    ptx::pdl_launch_dependents();
    const int64_t i0 = blockIdx.x * int64_t(THREADS * UNROLL_OUT) + threadIdx.x;
    uint32_t codes[UNROLL_OUT], s[UNROLL_OUT];
#pragma unroll
    for (int r = 0; r < UNROLL_OUT; ++r) {
        const int64_t i = i0 + r * THREADS;
        codes[r] = i < pieces ? reinterpret_cast<const Codes *>(q)[i] : 0u;
        s[r] = i < pieces ? sf[i / (32 / W)] : 0u;
    }
#pragma unroll
    for (int r = 0; r < UNROLL_OUT; ++r) {
        const int64_t i = i0 + r * THREADS;
        if (i >= pieces) break;
        // 2^(s - 127): code 0 is the subnormal 2^-127, 255 is NaN
        const float scale = __uint_as_float(s[r] == 0u ? 0x00400000u : s[r] == 255u ? 0x7FC00000u : s[r] << 23);
        float v[W];
#pragma unroll
        for (int u = 0; u < W; ++u) v[u] = __fmul_rn(e2m1_value(codes[r] >> (4 * u)), scale);
        store16(out + i * W, v);
    }
}

qgmm_status check_rows(int64_t rows, int64_t k, int32_t type)
{
    if (type != QGMM_T_BF16 && type != QGMM_T_F16 && type != QGMM_T_F32) return QGMM_ERR_DTYPE;
    if (rows < 0 || rows > (int64_t(1) << 31) - 1 || k < 32 || k > 65536 || k % 32) return QGMM_ERR_SHAPE;
    if (rows > (int64_t(1) << 42) / k) return QGMM_ERR_SHAPE;
    return QGMM_OK;
}

bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Launch on `pieces` of the tensor, `unroll` a thread, a block's side by side (blocks that take
// turns over the whole tensor were slower: 205 against 174 us for both kernels at
// 57344 x 2048 f32).  The kernel may start beside the one before it on the stream and waits
// for that one's results itself.
template <typename... P, typename... A>
qgmm_status launch(void (*kern)(P...), int unroll, int64_t pieces, void *cuda_stream, A... args)
{
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
        return QGMM_ERR_CUDA;
    if (major != 10) return QGMM_ERR_UNSUPPORTED;
    const int64_t block = THREADS * int64_t(unroll), blocks = (pieces + block - 1) / block;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess ? QGMM_OK : QGMM_ERR_CUDA;
}

}  // namespace
}  // namespace qgmm

using namespace qgmm;

QGMM_MM_API qgmm_status qgmm_per_token_quant_mxfp4(const void *x, int32_t x_type, int64_t rows, int64_t k,
                                                   uint8_t *q_out, uint8_t *sf_out, void *cuda_stream)
{
    qgmm_status s = check_rows(rows, k, x_type);
    if (s != QGMM_OK) return s;
    if (rows == 0) return QGMM_OK;
    if (!x || !q_out || !sf_out) return QGMM_ERR_NULL_PTR;
    if (misaligned(x, 16) || misaligned(q_out, 4)) return QGMM_ERR_ALIGNMENT;
    const int64_t eighths = rows * (k / 8);
    uint32_t *q = reinterpret_cast<uint32_t *>(q_out);
    switch (x_type) {
    case QGMM_T_BF16:
        return launch(quant_mxfp4_kernel<__nv_bfloat16>, UNROLL, eighths, cuda_stream, static_cast<const __nv_bfloat16 *>(x),
                      eighths, q, sf_out);
    case QGMM_T_F16:
        return launch(quant_mxfp4_kernel<__half>, UNROLL, eighths, cuda_stream, static_cast<const __half *>(x), eighths, q,
                      sf_out);
    default:
        return launch(quant_mxfp4_kernel<float>, UNROLL, eighths, cuda_stream, static_cast<const float *>(x), eighths, q,
                      sf_out);
    }
}

QGMM_MM_API qgmm_status qgmm_mxfp4_dequant(const uint8_t *q, const uint8_t *sf, int64_t rows, int64_t k, void *out,
                                           int32_t out_type, void *cuda_stream)
{
    qgmm_status s = check_rows(rows, k, out_type);
    if (s != QGMM_OK) return s;
    if (rows == 0) return QGMM_OK;
    if (!q || !sf || !out) return QGMM_ERR_NULL_PTR;
    if (misaligned(out, 16) || misaligned(q, 4)) return QGMM_ERR_ALIGNMENT;
    const int64_t eighths = rows * (k / 8), fourths = 2 * eighths;
    switch (out_type) {
    case QGMM_T_BF16:
        return launch(dequant_mxfp4_kernel<__nv_bfloat16>, UNROLL_OUT, eighths, cuda_stream, q, sf, eighths,
                      static_cast<__nv_bfloat16 *>(out));
    case QGMM_T_F16:
        return launch(dequant_mxfp4_kernel<__half>, UNROLL_OUT, eighths, cuda_stream, q, sf, eighths, static_cast<__half *>(out));
    default:
        return launch(dequant_mxfp4_kernel<float>, UNROLL_OUT, fourths, cuda_stream, q, sf, fourths, static_cast<float *>(out));
    }
}
