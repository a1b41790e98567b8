// grouped.cuh -- device helpers of the grouped products: the table of
// groups a CTA builds from the offsets, and typed loads and stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace strata {

// The groups as a CTA sees them: first row, rows, and the exclusive prefix
// sum of their row blocks (pre[E] = all blocks).  Offsets that run backwards
// anywhere or leave [0, M] make every group empty (STRATA_EBADROUTE is
// latched): the groups of a table are then always disjoint and in order, so
// their blocks fit the scales' buffers.
// of[b]: the group of row block b, for the first kBlockMap blocks.
constexpr int kBlockMap = 2048;
struct GroupTable {
    int row[kMaxExperts];
    int cnt[kMaxExperts];
    int pre[kMaxExperts + 1];
    int part[32];
    uint16_t of[kBlockMap];
};

// Built by all threads of the CTA (a multiple of 32, at most 1024); ends
// with a barrier.  offsets NULL: E equal groups of M / E rows.
__device__ __forceinline__ void build_groups(GroupTable& t, const int32_t* offsets, int E, int M,
                                             int block_rows, uint32_t* err) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad = false;
    for (int e = tid; e < E; e += int(blockDim.x)) {
        int row = e * (M / E), cnt = M / E;
        if (offsets != nullptr) {
            row = offsets[e];
            const int end = offsets[e + 1];
            bad |= row < 0 || end < row || end > M;
            cnt = end - row;
        }
        t.row[e] = row;
        t.cnt[e] = cnt;
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) latch(err, STRATA_EBADROUTE);
    int carry = 0;
    for (int base = 0; base < E; base += int(blockDim.x)) {
        const int e = base + tid;
        if (bad && e < E) t.row[e] = t.cnt[e] = 0;
        const int n = e < E ? (t.cnt[e] + block_rows - 1) / block_rows : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) t.part[warp] = incl;
        __syncthreads();
        int before = carry, all = carry;
        for (int w = 0; w < int(blockDim.x) >> 5; ++w) {
            if (w < warp) before += t.part[w];
            all += t.part[w];
        }
        const int first = before + incl - n;
        if (e < E) t.pre[e] = first;
        for (int b = first; b < min(first + n, kBlockMap); ++b) t.of[b] = uint16_t(e);
        carry = all;
        __syncthreads();
    }
    if (tid == 0) t.pre[E] = carry;
    __syncthreads();
}

// The group that holds row block b (b < pre[E]): from the map, or past it the
// last e with pre[e] <= b, which is not empty.
__device__ __forceinline__ int group_of_block(const GroupTable& t, int E, int b) {
    if (b < kBlockMap) return t.of[b];
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.pre[mid] <= b) lo = mid; else hi = mid;
    }
    return lo;
}

// Where row `r` lies: its group's rows [first, end) and first row block, or
// first = -1 for a row of no group (end = the next row that may have one).
// Computed by a whole warp straight from the offsets: a warp works on
// consecutive rows, so it looks a group up about once, and no table has to be
// built by the CTA before the first row is read.
struct RowGroup {
    int first, end, block, e;
};
__device__ __forceinline__ RowGroup row_group(const int32_t* offsets, int E, int rows, int r,
                                              uint32_t* err) {
    if (offsets == nullptr) {
        const int n = rows / E, e = r / n;
        return RowGroup{e * n, (e + 1) * n, e * ((n + 127) / 128), e};
    }
    int block = 0, first = -1, end = -1, group = -1;
    bool bad = false;
    for (int e = int(threadIdx.x & 31); e < E; e += 32) {
        const int a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
        bad |= a < 0 || b < a || b > rows;
        if (b <= r) {
            block += (b - a + 127) / 128;
        } else if (a <= r) {
            first = a;
            end = b;
            group = e;
        }
    }
    if (__any_sync(0xffffffffu, bad)) {
        if ((threadIdx.x & 31) == 0) latch(err, STRATA_EBADROUTE);
        return RowGroup{-1, rows, 0, -1};
    }
    block = __reduce_add_sync(0xffffffffu, block);
    first = __reduce_max_sync(0xffffffffu, first);
    end = __reduce_max_sync(0xffffffffu, end);
    if (first < 0) {
        const int o0 = __ldg(offsets);
        return RowGroup{-1, r < o0 ? o0 : rows, 0, -1};
    }
    return RowGroup{first, end, block, __reduce_max_sync(0xffffffffu, group)};
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// One rounding, to nearest even, from the fp32 sum to the output's type.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

}  // namespace strata
