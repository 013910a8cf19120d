// grouped_mm.cuh -- kernels of the grouped products: plain tiled f32 multiply-adds, one
// 64 x 64 output tile per block at a time, 4 x 4 outputs per thread.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "groups.cuh"

namespace qgmm {

constexpr int MM_MAX_E = 1024;
constexpr int MM_T = 64;    // output tile
constexpr int MM_K = 16;    // summed elements per step

struct E2M1 { uint8_t pair; };

struct MmArgs {
    const int64_t *group_list;
    int64_t m;
    int32_t e, group_list_type;
    const void *a, *w;
    const uint8_t *sfa, *sfw;
    void *out;
    uint32_t *status;
    int32_t c, j;              // rows: summed and output widths; wgrad: dw's rows and columns
    int64_t lda, ldo;
    int64_t w_group, w_c, w_j; // wgrad: w_group is dw's group stride, w_c the second operand's row stride
    int32_t accumulate;
};

__device__ __forceinline__ float mm_get(const __nv_bfloat16 *p, const uint8_t *, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float mm_get(const __half *p, const uint8_t *, int64_t i) { return __half2float(p[i]); }
__device__ __forceinline__ float mm_get(const E2M1 *p, const uint8_t *sf, int64_t i)
{
    const uint32_t c = (p[i >> 1].pair >> (4 * (i & 1))) & 15u, mag = c & 7u;
    const float v = mag < 4 ? 0.5f * mag : mag < 6 ? mag - 2.f : 2.f * mag - 8.f;
    const uint32_t s = sf[i >> 5];
    return (c & 8u ? -v : v) * __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7FC00000u : s << 23);
}
__device__ __forceinline__ void mm_put(float *p, float v) { *p = v; }
__device__ __forceinline__ void mm_put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void mm_put(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ float mm_old(const float *p) { return *p; }
__device__ __forceinline__ float mm_old(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float mm_old(const __half *p) { return __half2float(*p); }

__device__ __forceinline__ void mm_step(const float (&sa)[MM_K][MM_T + 1], const float (&sb)[MM_K][MM_T + 1],
                                        float (&acc)[4][4])
{
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int q = 0; q < MM_K; ++q)
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[u][v] += sa[q][ty + 16 * u] * sb[q][tx + 16 * v];
}

template <typename T, typename O>
__global__ void __launch_bounds__(256) mm_rows_kernel(const MmArgs p)
{
    __shared__ int32_t off[MM_MAX_E + 1], cum[MM_MAX_E + 1];
    __shared__ float sa[MM_K][MM_T + 1], sb[MM_K][MM_T + 1];
    if (threadIdx.x < 32) {
        const uint32_t f = decode_groups_warp(
            p.group_list, p.e, p.group_list_type, p.m,
            [](int64_t rows) { return static_cast<int32_t>((rows + MM_T - 1) / MM_T); }, off, cum);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = f;
    }
    __syncthreads();
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int nt = (p.j + MM_T - 1) / MM_T;
    const T *a = static_cast<const T *>(p.a), *w = static_cast<const T *>(p.w);
    for (int64_t t = blockIdx.x; t < int64_t(cum[p.e]) * nt; t += gridDim.x) {
        const int mt = static_cast<int>(t / nt), j0 = static_cast<int>(t % nt) * MM_T;
        int g = 0, hi = p.e;
        while (hi - g > 1) {
            const int mid = (g + hi) >> 1;
            if (cum[mid] <= mt) g = mid;
            else hi = mid;
        }
        const int r0 = off[g] + (mt - cum[g]) * MM_T, r1 = off[g + 1];
        float acc[4][4] = {};
        for (int c0 = 0; c0 < p.c; c0 += MM_K) {
            for (int i = threadIdx.x; i < MM_K * MM_T; i += 256) {
                const int q = i % MM_K, r = i / MM_K, c = c0 + q;
                sa[q][r] = c < p.c && r0 + r < r1 ? mm_get(a, p.sfa, int64_t(r0 + r) * p.lda + c) : 0.f;
                sb[q][r] = c < p.c && j0 + r < p.j
                               ? mm_get(w, p.sfw, int64_t(g) * p.w_group + int64_t(c) * p.w_c + int64_t(j0 + r) * p.w_j)
                               : 0.f;
            }
            __syncthreads();
            mm_step(sa, sb, acc);
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int r = r0 + ty + 16 * u, j = j0 + tx + 16 * v;
                if (r < r1 && j < p.j) mm_put(static_cast<O *>(p.out) + int64_t(r) * p.ldo + j, acc[u][v]);
            }
    }
}

template <typename T, typename O>
__global__ void __launch_bounds__(256) mm_wgrad_kernel(const MmArgs p)
{
    __shared__ int32_t off[MM_MAX_E + 1], cum[MM_MAX_E + 1];
    __shared__ float sa[MM_K][MM_T + 1], sb[MM_K][MM_T + 1];
    if (threadIdx.x < 32) {
        const uint32_t f = decode_groups_warp(
            p.group_list, p.e, p.group_list_type, p.m, [](int64_t) { return 0; }, off, cum);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = f;
    }
    __syncthreads();
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int ct = (p.c + MM_T - 1) / MM_T, jt = (p.j + MM_T - 1) / MM_T;
    const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.w);
    for (int64_t t = blockIdx.x; t < int64_t(p.e) * ct * jt; t += gridDim.x) {
        const int g = static_cast<int>(t / (ct * jt)), r = static_cast<int>(t % (ct * jt));
        const int c0 = r / jt * MM_T, j0 = r % jt * MM_T;
        if (p.accumulate && off[g] == off[g + 1]) continue;
        float acc[4][4] = {};
        for (int i0 = off[g]; i0 < off[g + 1]; i0 += MM_K) {
            for (int i = threadIdx.x; i < MM_K * MM_T; i += 256) {
                const int q = i / MM_T, x = i % MM_T, row = i0 + q;
                sa[q][x] = row < off[g + 1] && c0 + x < p.c ? mm_get(a, nullptr, int64_t(row) * p.lda + c0 + x) : 0.f;
                sb[q][x] = row < off[g + 1] && j0 + x < p.j ? mm_get(b, nullptr, int64_t(row) * p.w_c + j0 + x) : 0.f;
            }
            __syncthreads();
            mm_step(sa, sb, acc);
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int c = c0 + ty + 16 * u, j = j0 + tx + 16 * v;
                if (c >= p.c || j >= p.j) continue;
                O *o = static_cast<O *>(p.out) + int64_t(g) * p.w_group + int64_t(c) * p.ldo + j;
                mm_put(o, p.accumulate ? mm_old(o) + acc[u][v] : acc[u][v]);
            }
    }
}

}  // namespace qgmm
