// grouped_simt.cuh -- the grouped products on the CUDA cores, for widths that
// the tensor maps cannot address.  EPI takes four columns of an output row at a
// time: epi(row, first column, values, whether the row exists).
#pragma once

#include "grouped.cuh"
#include "grouped.h"

namespace strata {

constexpr int kSimtTile = 64, kSimtK = 16, kSimtThreads = 256;
// Terms of a partial sum.  Added one by one, 2^18 equal terms came out 2e-3
// off: within a binade all their roundings go one way.
constexpr int kSimtPiece = 512;

// The sums as the output's type.
template <typename TO>
struct SimtStore {
    TO* out;
    int cols;
    __device__ __forceinline__ void operator()(size_t row, int c, const float* v, bool live) const {
        if (!live) return;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < cols) out[row * cols + c + j] = from_f32<TO>(v[j]);
    }
};

// One 64 x 64 output tile a CTA step, 4 x 4 outputs a thread, operands
// through shared memory as fp32.  For widths whose rows TMA cannot address (not
// a multiple of 16 bytes); bound by shared memory and FMAs, far from the tensor
// cores: 1024 rows of 8 experts, 1023 to 1024 columns, 204 us (1024 columns, on
// the tensor cores: 8.3), their dw over 8192 rows 868 (17).
template <int MODE, typename TI, typename EPI>
__global__ void __launch_bounds__(kSimtThreads) k_gmm_simt(GmmArgs g, EPI epi) {
    __shared__ GroupTable t;
    __shared__ float as[kSimtK][kSimtTile + 4], bs[kSimtK][kSimtTile + 4];
    build_groups(t, g.offsets, g.E, g.M, kSimtTile, g.err);
    const TI* A = static_cast<const TI*>(g.a);
    const TI* B = static_cast<const TI*>(g.b);
    const int cols = MODE == kGmmFwd ? g.N : g.K;
    const int nt = (cols + kSimtTile - 1) / kSimtTile;
    const int mt = (g.N + kSimtTile - 1) / kSimtTile;        // dw: row tiles of one expert
    const long long tiles = MODE == kGmmDw ? (long long)g.E * mt * nt : (long long)t.pre[g.E] * nt;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int c0 = int(tile % nt) * kSimtTile;
        const int rb = int(tile / nt);
        int e, row0, rows, red, a0 = 0;
        if (MODE == kGmmDw) {
            e = rb / mt;
            row0 = (rb % mt) * kSimtTile;                      // row of W[e]
            rows = min(kSimtTile, g.N - row0);
            red = t.cnt[e];
            a0 = t.row[e];
        } else {
            e = group_of_block(t, g.E, rb);
            const int in = (rb - t.pre[e]) * kSimtTile;
            row0 = t.row[e] + in;
            rows = min(kSimtTile, t.cnt[e] - in);
            red = MODE == kGmmFwd ? g.K : g.N;
        }
        float sum[4][4] = {}, acc[4][4] = {};
        auto join = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[i][j] += acc[i][j];
                    acc[i][j] = 0.0f;
                }
        };
        for (int k0 = 0; k0 < red; k0 += kSimtK) {
            if (k0 % kSimtPiece == 0) join();
            __syncthreads();
            for (int i = threadIdx.x; i < kSimtTile * kSimtK; i += kSimtThreads) {
                // the lane order follows memory: along k, or along the tile where
                // the operand's rows run along the reduction
                int r, k;
                if (MODE == kGmmDw) { r = i % kSimtTile; k = i / kSimtTile; }
                else { k = i % kSimtK; r = i / kSimtK; }
                const bool in_k = k0 + k < red;
                float v = 0.0f;
                if (in_k && r < rows) {
                    if (MODE == kGmmDw) v = to_f32(A[size_t(a0 + k0 + k) * g.N + row0 + r]);
                    else v = to_f32(A[size_t(row0 + r) * red + k0 + k]);
                }
                as[k][r] = v;
                if (MODE != kGmmFwd) { r = i % kSimtTile; k = i / kSimtTile; }
                v = 0.0f;
                if (k0 + k < red && c0 + r < cols) {
                    if (MODE == kGmmFwd) v = to_f32(B[(size_t(e) * g.N + c0 + r) * g.K + k0 + k]);
                    else if (MODE == kGmmDx)
                        v = to_f32(B[(size_t(e) * g.N + k0 + k) * g.K + c0 + r]);
                    else v = to_f32(B[size_t(a0 + k0 + k) * g.K + c0 + r]);
                }
                bs[k][r] = v;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kSimtK; ++k) {
                float av[4], bv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    av[i] = as[k][ty * 4 + i];
                    bv[i] = bs[k][tx * 4 + i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
            }
        }
        join();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            const size_t at = MODE == kGmmDw ? size_t(e) * g.N + row0 + r : size_t(row0 + r);
            epi(at, c0 + tx * 4, sum[i], r < rows);
        }
    }
}

}  // namespace strata
