// grouped_few.cuh -- the forward product for a handful of rows (the slots of
// one token): every touched expert's W is streamed through the CUDA cores.
// The tensor-core kernel takes a reduction of 2048 as 32 pipeline stages in a
// row, each a quarter of a microsecond however few rows there are; here all of
// a warp's loads are in flight at once.
//
// Measured (1024 x 2048 experts, bf16, 8 rows of 8 experts, 33.5 MB, another
// eight every call so that they come from HBM): 7.6 us (4.4 TB/s; 5.3 where the
// L2 holds them) against 11.4 on the tensor cores; 16 rows of 16: 13.0 against
// 15.2; 32 rows of 4 experts: 12.2 against 14.3, but from the L2 11.6 against
// 10.3.  Hence at most 8 rows, where both favour it.
//
// Every CTA finds the touched groups itself (one load of the offsets), then
// the warps of the grid take (group, rows of W) units in turn.  A lane loads
// 16 bytes of several W rows at once; the row's sum is closed by shuffles, so
// its order is fixed.  A lane's sum is set aside every 8192 columns: one by
// one, equal terms of a reduction of 2^20 came out 4e-4 off, as within a
// binade all their roundings go one way.
#pragma once

#include "grouped.cuh"
#include "grouped.h"

namespace strata {

namespace {

constexpr int kFewThreads = 256;
constexpr int kFewX = 4;                 // x rows a pass over W serves

// The touched groups, keyed by their first row.
struct FewTable {
    uint32_t mask;                       // bit r: a group starts at row r
    int e[kFewRowsMax], cnt[kFewRowsMax];
    int row[kFewRowsMax];                // the touched groups' first rows, in order
};
static_assert(kFewRowsMax <= 32, "rows in a word");
// Returns their number.
__device__ __forceinline__ int few_groups(FewTable& t, const int32_t* offsets, int E, int M,
                                               uint32_t* err) {
    if (threadIdx.x == 0) t.mask = 0u;
    __syncthreads();
    bool bad = false;
    for (int e = threadIdx.x; e < E; e += kFewThreads) {
        const int a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
        if (a < 0 || b < a || b > M) {
            bad = true;
        } else if (b > a) {
            atomicOr(&t.mask, 1u << a);
            t.e[a] = e;
            t.cnt[a] = b - a;
        }
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) latch(err, STRATA_EBADROUTE);
    const uint32_t mask = bad ? 0u : t.mask;
    const int r = threadIdx.x;
    if (r < kFewRowsMax && (mask >> r & 1u)) t.row[__popc(mask & ((1u << r) - 1u))] = r;
    __syncthreads();
    return __popc(mask);
}

// c + a b for the two halves of packed 16-bit words, products exact in fp32.
template <bool BF16>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    if (BF16) return fma_bf16<true, true>(a, b, fma_bf16<false, false>(a, b, c));
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    return fmaf(fa.y, fb.y, fmaf(fa.x, fb.x, c));
}
template <bool BF16>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float c) {
    return dot2<BF16>(a.w, b.w, dot2<BF16>(a.z, b.z, dot2<BF16>(a.y, b.y, dot2<BF16>(a.x, b.x, c))));
}

constexpr int kFewRows = 4;              // W rows a warp works on (16-bit operands)
constexpr int kFewLoads = 4;             // 16-byte pieces of each a lane has in flight
constexpr int kFewChunk = 1024;          // 16-byte pieces of a row between two such sums
// The kernels of longer rows are their own (LONG): the checks alone cost the
// others 3 to 6 % (8 rows of 2048: 5.25 and 5.4 us).
inline bool few_long(const GmmArgs& g) { return g.K > kFewChunk * 8; }

// X rows of x (row ..) by kFewRows rows of W (n0 ..); EPI takes their sums,
// which all lanes have: epi(row, n0, sums).
// aside (LONG): X x kFewRows x 32 floats of the warp's own.
template <int X, bool BF16, bool LONG, typename EPI>
__device__ __forceinline__ void few_unit(const GmmArgs& g, const EPI& epi, int e, int n0, int row,
                                         float* aside) {
    const int lane = threadIdx.x & 31, pieces = g.K / 8;     // 16-byte pieces of a row
    const uint4* x = static_cast<const uint4*>(g.a) + size_t(row) * pieces;
    const uint4* w = static_cast<const uint4*>(g.b) + size_t(e) * g.N * pieces;
    const uint4* wr[kFewRows];
#pragma unroll
    for (int i = 0; i < kFewRows; ++i) wr[i] = w + size_t(min(n0 + i, g.N - 1)) * pieces;
    float acc[X][kFewRows] = {};
    for (int p0 = lane; p0 < pieces; p0 += 32 * kFewLoads) {
        if (LONG && p0 >= kFewChunk && p0 % kFewChunk == lane) {
#pragma unroll
            for (int r = 0; r < X; ++r)
#pragma unroll
                for (int i = 0; i < kFewRows; ++i) {
                    float* t = aside + (r * kFewRows + i) * 32 + lane;
                    *t = p0 == kFewChunk + lane ? acc[r][i] : *t + acc[r][i];
                    acc[r][i] = 0.0f;
                }
        }
        uint4 v[kFewRows][kFewLoads];
#pragma unroll
        for (int l = 0; l < kFewLoads; ++l)
#pragma unroll
            for (int i = 0; i < kFewRows; ++i)
                v[i][l] = p0 + 32 * l < pieces ? ldg_stream(wr[i] + p0 + 32 * l)
                                               : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int l = 0; l < kFewLoads; ++l) {
            // past the row's end neither operand is read: the accumulators stay
            if (p0 + 32 * l >= pieces) break;
#pragma unroll
            for (int r = 0; r < X; ++r) {
                const uint4 xv = __ldg(x + size_t(r) * pieces + p0 + 32 * l);
#pragma unroll
                for (int i = 0; i < kFewRows; ++i) acc[r][i] = dot8<BF16>(v[i][l], xv, acc[r][i]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < X; ++r) {
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) {
            // what a lane has set aside is its own
            if (LONG && pieces > kFewChunk + lane) acc[r][i] += aside[(r * kFewRows + i) * 32 + lane];
            acc[r][i] = warp_sum(acc[r][i]);
        }
        epi(size_t(row + r), n0, acc[r]);
    }
}

// CTAS: blocks an SM.  Two leave a thread 128 registers and spill a few; a grid
// that has no more than one an SM keeps them all (us, bf16 and fp16, two and one:
// 8 rows of 2 experts, 512 x 1032, 6.8 7.3 and 5.7 5.8; of 8 experts, 512 x 2048,
// 6.0 6.2 and 5.8 5.9; but 1024 x 2048, whose grid is larger, 7.7 7.9 and 9.3 9.5).
template <bool BF16, bool LONG, int CTAS, typename EPI>
__global__ void __launch_bounds__(kFewThreads, CTAS) k_gmm_few(GmmArgs g, EPI epi) {
    __shared__ FewTable t;
    __shared__ float aside[LONG ? kFewThreads / 32 : 1][LONG ? kFewX * kFewRows * 32 : 1];
    pdl_launch();
    pdl_wait();
    float* own = aside[LONG ? threadIdx.x >> 5 : 0];
    const int chunks = (g.N + kFewRows - 1) / kFewRows;
    const int units = few_groups(t, g.offsets, g.E, g.M, g.err) * chunks;
    for (int u = int(blockIdx.x * (kFewThreads / 32) + (threadIdx.x >> 5)); u < units;
         u += int(gridDim.x) * (kFewThreads / 32)) {
        const int row = t.row[u / chunks], n0 = (u % chunks) * kFewRows;
        const int e = t.e[row], cnt = t.cnt[row];
        int r = 0;
        for (; r + kFewX <= cnt; r += kFewX) few_unit<kFewX, BF16, LONG>(g, epi, e, n0, row + r, own);
        for (; r < cnt; ++r) few_unit<1, BF16, LONG>(g, epi, e, n0, row + r, own);
    }
}

template <typename... P, typename... A>
cudaError_t few_launch(void (*kernel)(P...), int units, int per_sm, cudaStream_t s,
                       const A&... args) {
    const int want = (units + kFewThreads / 32 - 1) / (kFewThreads / 32);
    const int most = device_info().sms * per_sm;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(want < most ? want : most);
    cfg.blockDim = dim3(kFewThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool BF16, typename EPI>
cudaError_t run_few(const GmmArgs& g, const EPI& epi, cudaStream_t s) {
    const int units = (g.M < g.E ? g.M : g.E) * ((g.N + kFewRows - 1) / kFewRows);
    if (units <= device_info().sms * (kFewThreads / 32))
        return few_long(g) ? few_launch(k_gmm_few<BF16, true, 1, EPI>, units, 1, s, g, epi)
                           : few_launch(k_gmm_few<BF16, false, 1, EPI>, units, 1, s, g, epi);
    return few_long(g) ? few_launch(k_gmm_few<BF16, true, 2, EPI>, units, 2, s, g, epi)
                       : few_launch(k_gmm_few<BF16, false, 2, EPI>, units, 2, s, g, epi);
}

}  // namespace

}  // namespace strata
