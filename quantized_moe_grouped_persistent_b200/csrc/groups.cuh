// groups.cuh -- the group list, as every grouped kernel of this package reads it.
#pragma once

#include <cstdint>

#include "../../include/qgmm.h"

namespace qgmm {

// ---------------------------------------------------------------- groups
// Warp-cooperative decode of groupList (page 1, parameter constraints):
// off[g+1] = end row of group g, cum[g+1] = m-tiles of groups 0..g.
// Invalid lists are sanitised so every offset stays in [0, m] and monotone
// (type 0: running max of clamp(end, 0, m); type 1: clamp of the running sum
// of max(count, 0)); the returned QGMM_DEV_* bits say what was wrong.
// tiles_of(rows) gives the m-tiles of a group of `rows` rows.
template <typename TilesOf>
__device__ __forceinline__ uint32_t decode_groups_warp(const int64_t *gl, int e, int type, int64_t m,
                                                       TilesOf tiles_of, int32_t *off, int32_t *cum)
{
    const int lane = threadIdx.x & 31;
    uint32_t flags = 0;
    int64_t carry_end = 0;     // end of the previous chunk's last group
    int64_t carry_sum = 0;     // type 1: unclamped running sum
    int32_t carry_cum = 0;
    if (lane == 0) {
        off[0] = 0;
        cum[0] = 0;
    }
    for (int base = 0; base < e; base += 32) {
        const int g = base + lane;
        const bool in = g < e;
        const int64_t v = in ? gl[g] : 0;
        if (in && v < 0) flags |= QGMM_DEV_GROUP_NEGATIVE;
        int64_t end;
        if (type == 0) {
            if (in && g > 0 && v < gl[g - 1]) flags |= QGMM_DEV_GROUP_NOT_MONOTONE;
            if (in && v > m) flags |= QGMM_DEV_GROUP_TOTAL_GT_M;
            int64_t s = v < 0 ? 0 : (v > m ? m : v);
            if (!in) s = 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d && o > s) s = o;
            }
            end = s > carry_end ? s : carry_end;
        } else {
            int64_t s = (in && v > 0) ? (v > m ? m + 1 : v) : 0;   // past m it only has to stay past m
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += o;
            }
            s += carry_sum;
            carry_sum = __shfl_sync(0xffffffffu, s, 31);
            if (in && s > m) flags |= QGMM_DEV_GROUP_TOTAL_GT_M;
            end = s > m ? m : s;
        }
        int64_t start = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) start = carry_end;
        const int64_t rows = end - start;
        int32_t mt = in ? tiles_of(rows) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, mt, d);
            if (lane >= d) mt += o;
        }
        mt += carry_cum;
        if (in) {
            off[g + 1] = static_cast<int32_t>(end);
            cum[g + 1] = mt;
        }
        carry_end = __shfl_sync(0xffffffffu, end, 31);
        carry_cum = __shfl_sync(0xffffffffu, mt, 31);
    }
    // OR-reduce the flags across the warp
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) flags |= __shfl_xor_sync(0xffffffffu, flags, d);
    __syncwarp();
    return flags;
}

}  // namespace qgmm
