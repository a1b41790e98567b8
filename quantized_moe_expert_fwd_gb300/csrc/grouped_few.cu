// grouped_few.cu -- the forward product for a handful of rows (the slots of
// one token) or of columns.  Rows: every touched expert's W is streamed through the CUDA cores.
// The tensor-core kernel takes a reduction of 2048 as 32 pipeline stages in a
// row, each a quarter of a microsecond however few rows there are; here all of
// a warp's loads are in flight at once.
//
// Measured (1024 x 2048 experts, bf16, 8 rows of 8 experts, 33.5 MB): 6.5 us
// (5.1 TB/s) against 11.1 on the tensor cores; 16 rows: 13.8 against 14.0;
// 32 rows of 4 experts: 11.6 against 10.3.  Hence at most 8 rows.
//
// Every CTA finds the touched groups itself (one load of the offsets), then
// the warps of the grid take (group, rows of W) units in turn.  A lane loads
// 16 bytes of several W rows at once; the row's sum is closed by shuffles, so
// its order is fixed.  A lane's sum is set aside every 8192 columns: one by
// one, equal terms of a reduction of 2^20 came out 4e-4 off, as within a
// binade all their roundings go one way.
#include "grouped.cuh"
#include "grouped.h"

namespace strata {

namespace {

constexpr int kFewThreads = 256;
constexpr int kFewX = 4;                 // x rows a pass over W serves
constexpr int kNarrowCols = kNarrowColsMax;

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

// X rows of x (row ..) by kFewRows rows of W.
// aside (LONG): X x kFewRows x 32 floats of the warp's own.
template <int X, bool BF16, bool LONG, typename TO>
__device__ __forceinline__ void few_unit(const GmmArgs& g, int e, int n0, int row, float* aside) {
    const int lane = threadIdx.x & 31, pieces = g.K / 8;     // 16-byte pieces of a row
    const uint4* x = static_cast<const uint4*>(g.a) + size_t(row) * pieces;
    const uint4* w = static_cast<const uint4*>(g.b) + size_t(e) * g.N * pieces;
    TO* y = static_cast<TO*>(g.out) + size_t(row) * g.N;
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
    for (int r = 0; r < X; ++r)
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) {
            // what a lane has set aside is its own
            if (LONG && pieces > kFewChunk + lane) acc[r][i] += aside[(r * kFewRows + i) * 32 + lane];
            const float s = warp_sum(acc[r][i]);
            if (lane == i && n0 + i < g.N) y[size_t(r) * g.N + n0 + i] = from_f32<TO>(s);
        }
}

template <bool BF16, bool LONG, typename TO>
__global__ void __launch_bounds__(kFewThreads) k_gmm_few(GmmArgs g) {
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
        for (; r + kFewX <= cnt; r += kFewX) few_unit<kFewX, BF16, LONG, TO>(g, e, n0, row + r, own);
        for (; r < cnt; ++r) few_unit<1, BF16, LONG, TO>(g, e, n0, row + r, own);
    }
}

// Few columns instead of few rows: a warp a row of x, every column's W row
// from the caches (the warps of a CTA work on neighbouring rows, so mostly on
// one expert's).  On the tensor cores a tile of any width takes every stage of
// the reduction.  Tensor cores and here, us, calls back to back: 2536 rows of
// 317 experts, 1816 wide, 1 column 24.2 4.4, 4 columns 24.3 6.6, 8 columns 24.0
// 9.3; 8000 rows of 4 experts, 4096 wide (in the L2), 21.7 9.3, 17.2 19.5, 16.4
// 33.1; 32000 such rows, 62.0 41.6, 46.0 58.2, 45.7 113.7.  Hence at most 4
// columns: 5 to 8 would gain only where the experts have few rows.
template <bool BF16, bool LONG, typename TO>
__global__ void __launch_bounds__(kFewThreads, 3) k_gmm_narrow(GmmArgs g) {
    pdl_launch();
    pdl_wait();
    const int lane = threadIdx.x & 31, pieces = g.K / 8;
    const int warps = int(gridDim.x) * (kFewThreads / 32);
    const int wi = int(blockIdx.x) * (kFewThreads / 32) + int(threadIdx.x >> 5);
    const uint4* w = static_cast<const uint4*>(g.b);
    TO* y = static_cast<TO*>(g.out);
    RowGroup gr{-1, -1, 0, -1};
    const int last = int((long long)g.M * (wi + 1) / warps);
    for (int row = int((long long)g.M * wi / warps); row < last; ++row) {
        if (row >= gr.end) gr = row_group(g.offsets, g.E, g.M, row, g.err);
        if (gr.first < 0) {
            row = gr.end - 1;
            continue;
        }
        const uint4* x = static_cast<const uint4*>(g.a) + size_t(row) * pieces;
        const uint4* we = w + size_t(gr.e) * g.N * pieces;
        float acc[kNarrowCols] = {}, aside[kNarrowCols] = {};
        for (int p0 = lane; p0 < pieces; p0 += 32 * kFewLoads) {
            if (LONG && p0 >= kFewChunk && p0 % kFewChunk == lane) {
#pragma unroll
                for (int n = 0; n < kNarrowCols; ++n) {
                    aside[n] += acc[n];
                    acc[n] = 0.0f;
                }
            }
            uint4 v[kFewLoads];
#pragma unroll
            for (int l = 0; l < kFewLoads; ++l)
                v[l] = p0 + 32 * l < pieces ? ldg_stream(x + p0 + 32 * l) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int n = 0; n < kNarrowCols; ++n) {
                if (n >= g.N) break;
#pragma unroll
                for (int l = 0; l < kFewLoads; ++l)
                    if (p0 + 32 * l < pieces)
                        acc[n] = dot8<BF16>(v[l], __ldg(we + size_t(n) * pieces + p0 + 32 * l), acc[n]);
            }
        }
#pragma unroll
        for (int n = 0; n < kNarrowCols; ++n) {
            if (n >= g.N) break;
            const float s = warp_sum(LONG ? aside[n] + acc[n] : acc[n]);
            if (lane == n) y[size_t(row) * g.N + n] = from_f32<TO>(s);
        }
    }
}

template <typename... P, typename A>
cudaError_t few_launch(void (*kernel)(P...), int units, int per_sm, cudaStream_t s,
                       const A& args) {
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
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

template <bool BF16, typename TO>
cudaError_t run_few(const GmmArgs& g, cudaStream_t s) {
    const int units = (g.M < g.E ? g.M : g.E) * ((g.N + kFewRows - 1) / kFewRows);
    return few_long(g) ? few_launch(k_gmm_few<BF16, true, TO>, units, 2, s, g)
                       : few_launch(k_gmm_few<BF16, false, TO>, units, 2, s, g);
}
template <bool BF16, typename TO>
cudaError_t run_narrow(const GmmArgs& g, cudaStream_t s) {
    return few_long(g) ? few_launch(k_gmm_narrow<BF16, true, TO>, g.M, 3, s, g)
                       : few_launch(k_gmm_narrow<BF16, false, TO>, g.M, 3, s, g);
}

}  // namespace

cudaError_t launch_grouped_few(const GmmArgs& g, cudaStream_t s) {
    if (g.dtype == STRATA_BF16)
        return g.out_dtype == STRATA_F32 ? run_few<true, float>(g, s)
                                         : run_few<true, __nv_bfloat16>(g, s);
    return g.out_dtype == STRATA_F32 ? run_few<false, float>(g, s) : run_few<false, __half>(g, s);
}

cudaError_t launch_grouped_narrow(const GmmArgs& g, cudaStream_t s) {
    if (g.dtype == STRATA_BF16)
        return g.out_dtype == STRATA_F32 ? run_narrow<true, float>(g, s)
                                         : run_narrow<true, __nv_bfloat16>(g, s);
    return g.out_dtype == STRATA_F32 ? run_narrow<false, float>(g, s)
                                     : run_narrow<false, __half>(g, s);
}

}  // namespace strata
