// grouped_mm.cu -- grouped products in bf16, fp16 and MXFP4 and the gradients of the
// 16-bit ones: argument checks, plans and launches for the C ABI in qgmm_mm.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/qgmm_mm.h"
#include "grouped_mm.cuh"

#define QGMM_MM_API extern "C" __attribute__((visibility("default")))

namespace qgmm {
namespace {

constexpr size_t kWsAlign = 256;
constexpr int64_t kMaxM = int64_t(1) << 24;

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

qgmm_status check_call(const qgmm_mm_problem *p, const void *group_list, const void *workspace, size_t ws_bytes)
{
    if (!group_list || !workspace) return QGMM_ERR_NULL_PTR;
    if (misaligned(workspace, kWsAlign)) return QGMM_ERR_ALIGNMENT;
    size_t need = 0;
    const qgmm_status s = qgmm_grouped_mm_workspace(p, &need);
    if (s != QGMM_OK) return s;
    return ws_bytes < need ? QGMM_ERR_WORKSPACE_TOO_SMALL : QGMM_OK;
}

qgmm_status sm_count(int *sms)
{
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
        return QGMM_ERR_CUDA;
    return major == 10 ? QGMM_OK : QGMM_ERR_UNSUPPORTED;
}

// One product over rows: out[i][j] = sum_c a[i][c] * w(g, c, j), w element (g, c, j) at
// w + g * w_group + c * w_c + j * w_j.
template <typename T>
qgmm_status launch_rows(const MmArgs &a, int32_t out_type, int sms, cudaStream_t st)
{
    const int grid = 4 * sms;
    if (out_type == QGMM_T_F32)
        mm_rows_kernel<T, float><<<grid, 256, 0, st>>>(a);
    else if (out_type == QGMM_T_BF16)
        mm_rows_kernel<T, __nv_bfloat16><<<grid, 256, 0, st>>>(a);
    else
        mm_rows_kernel<T, __half><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? QGMM_OK : QGMM_ERR_CUDA;
}

template <typename T>
qgmm_status launch_wgrad(const MmArgs &a, int32_t out_type, int sms, cudaStream_t st)
{
    const int grid = 4 * sms;
    if (out_type == QGMM_T_F32)
        mm_wgrad_kernel<T, float><<<grid, 256, 0, st>>>(a);
    else
        mm_wgrad_kernel<T, T><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? QGMM_OK : QGMM_ERR_CUDA;
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
    if (misaligned(x, 16) || misaligned(w, 16) || misaligned(out, 16)) return QGMM_ERR_ALIGNMENT;
    if (p->m == 0) return QGMM_OK;
    int sms = 0;
    if ((s = sm_count(&sms)) != QGMM_OK) return s;
    const int64_t ldw = ld_or(p->ld_w, p->transpose_w ? p->k : p->n);
    MmArgs a = {};
    a.group_list = group_list;
    a.group_list_type = p->group_list_type;
    a.e = static_cast<int32_t>(p->e);
    a.m = p->m;
    a.a = x;
    a.w = w;
    a.sfa = sfx;
    a.sfw = sfw;
    a.out = out;
    a.status = static_cast<uint32_t *>(workspace);
    a.c = static_cast<int32_t>(dgrad ? p->n : p->k);
    a.j = static_cast<int32_t>(dgrad ? p->k : p->n);
    a.lda = dgrad ? ld_or(p->ld_y, p->n) : ld_or(p->ld_x, p->k);
    a.ldo = dgrad ? ld_or(p->ld_x, p->k) : ld_or(p->ld_y, p->n);
    a.w_group = (p->transpose_w ? p->n : p->k) * ldw;
    const bool c_outer = (p->transpose_w != 0) == dgrad;   // the summed index selects w's row
    a.w_c = c_outer ? ldw : 1;
    a.w_j = c_outer ? 1 : ldw;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (mx) return launch_rows<E2M1>(a, p->out_type, sms, st);
    return p->x_type == QGMM_T_BF16 ? launch_rows<__nv_bfloat16>(a, p->out_type, sms, st)
                                    : launch_rows<__half>(a, p->out_type, sms, st);
}

}  // namespace
}  // namespace qgmm

using namespace qgmm;

QGMM_MM_API qgmm_status qgmm_grouped_mm_workspace(const qgmm_mm_problem *p, size_t *ws_bytes)
{
    if (!ws_bytes) return QGMM_ERR_NULL_PTR;
    const qgmm_status s = check_problem(p);
    if (s != QGMM_OK) return s;
    *ws_bytes = kWsAlign;
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
    int sms = 0;
    if ((s = sm_count(&sms)) != QGMM_OK) return s;
    // dw's rows are the dimension `a` covers, its columns the one `w` covers
    const bool t = p->transpose_w != 0;
    MmArgs a = {};
    a.group_list = group_list;
    a.group_list_type = p->group_list_type;
    a.e = static_cast<int32_t>(p->e);
    a.m = p->m;
    a.a = t ? dy : x;
    a.w = t ? x : dy;
    a.out = dw;
    a.status = static_cast<uint32_t *>(workspace);
    a.c = static_cast<int32_t>(t ? p->n : p->k);
    a.j = static_cast<int32_t>(t ? p->k : p->n);
    const int64_t ldx = ld_or(p->ld_x, p->k), ldy = ld_or(p->ld_y, p->n);
    a.lda = t ? ldy : ldx;
    a.w_c = t ? ldx : ldy;
    a.ldo = ld_or(p->ld_w, t ? p->k : p->n);
    a.w_group = a.c * a.ldo;
    a.accumulate = p->accumulate;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    return p->x_type == QGMM_T_BF16 ? launch_wgrad<__nv_bfloat16>(a, p->out_type, sms, st)
                                    : launch_wgrad<__half>(a, p->out_type, sms, st);
}
