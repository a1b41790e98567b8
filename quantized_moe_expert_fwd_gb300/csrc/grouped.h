// grouped.h -- host-side declarations of the grouped products by expert
// (grouped.cu) and of the 4-bit block formats (fp4.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace strata {

constexpr size_t kGroupedWsBytes = 65536;

enum GroupedMode { kGmmFwd = 0, kGmmDx = 1, kGmmDw = 2 };

// One grouped product.  Rows of the slot space [M]; group e holds rows
// offsets[e] .. offsets[e + 1].  w is [E][N][K].
//   kGmmFwd  a = x  [M][K], b = w,          out = y  [M][N]
//   kGmmDx   a = dy [M][N], b = w,          out = dx [M][K]
//   kGmmDw   a = dy [M][N], b = x [M][K],   out = dw [E][N][K]
struct GmmArgs {
    const void* a; const void* b;
    void* out;
    const int32_t* offsets;
    uint32_t* err;
    int M, K, N, E;
    int dtype, out_dtype;            // strata_dtype
};
cudaError_t launch_grouped_mm(GroupedMode mode, const GmmArgs& g, cudaStream_t s);
// The tensor-core kernels, and whether they take this shape.
bool grouped_tc_takes(GroupedMode mode, const GmmArgs& g);
// The forward product of at most kFewRowsMax rows on the CUDA cores.
constexpr int kFewRowsMax = 8;
cudaError_t launch_grouped_few(const GmmArgs& g, cudaStream_t s);
// The forward product of at most kNarrowColsMax columns, there too.
constexpr int kNarrowColsMax = 4;
cudaError_t launch_grouped_narrow(const GmmArgs& g, cudaStream_t s);
cudaError_t launch_grouped_tc(GroupedMode mode, const GmmArgs& g, cudaStream_t s);

// Scales of `rows` rows by `cols` columns in `groups` groups, in bytes:
// ragged groups (offsets on the device) get the most blocks they can need.
size_t fp4_scale_bytes(int fmt, int64_t rows, int64_t cols, int64_t groups, bool ragged);

struct Fp4QuantArgs {
    const void* x; int x_rows, dtype;
    const int32_t* perm; int top_k;  // source row perm[row] / top_k, or perm NULL: row
    uint8_t* q; uint8_t* scales;
    const int32_t* offsets;          // NULL: n_groups equal groups
    uint32_t* err;
    int rows, cols, n_groups, fmt, scale_exp;
};
cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, cudaStream_t s);

struct Fp4DequantArgs {
    const uint8_t* q; const uint8_t* scales;
    void* out; int out_dtype;
    const int32_t* offsets;
    uint32_t* err;
    int rows, cols, n_groups, fmt, scale_exp;
};
cudaError_t launch_fp4_dequantize(const Fp4DequantArgs& a, cudaStream_t s);

struct Fp4GmmArgs {
    const uint8_t* xq; const uint8_t* xs;
    const uint8_t* wq; const uint8_t* wsc;
    const float* alpha;              // [E] or NULL (1)
    void* out; int out_dtype;
    const int32_t* offsets;
    uint32_t* err;
    int M, K, N, E, fmt, swiglu;
};
cudaError_t launch_grouped_mm_fp4(const Fp4GmmArgs& g, cudaStream_t s);

}  // namespace strata
