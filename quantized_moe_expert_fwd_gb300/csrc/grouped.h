// grouped.h -- host-side declarations of the grouped products by expert
// (grouped.cu), of the 4-bit block formats (fp4.cu) and of a tuning step's
// operators around them (swiglu.cu, act8.cu, slots.cu, norm.cu).
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

// SwiGLU of x W^T (w [E][2I][K], gate and up rows interleaved); p kept where
// it is given, in dtype or (scales given) in 8 bits.
struct SwigluArgs {
    const void* x; const void* w;
    const int32_t* offsets;
    void* h; void* p; uint8_t* scales;
    uint32_t* err;
    int M, K, I, E, dtype;
};
cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t s);
// dp from dh = dy W (w [E][N][I]) and the kept p; h again where it is given.
struct SwigluBwdArgs {
    const void* dy; const void* w;
    const void* p; const uint8_t* scales;
    const int32_t* offsets;
    void* dp; void* h;
    uint32_t* err;
    int M, N, I, E, dtype;
};
cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t s);

struct Act8SaveArgs {
    const void* x; uint8_t* q; uint8_t* scales;
    int rows, cols, dtype;
};
cudaError_t launch_act8_save(const Act8SaveArgs& a, cudaStream_t s);
struct Act8LoadArgs {
    const uint8_t* q; const uint8_t* scales;
    const int32_t* perm; int top_k;  // source row perm[row] / top_k, or perm NULL: row
    void* out;
    uint32_t* err;
    int q_rows, rows, cols, out_dtype;
};
cudaError_t launch_act8_load(const Act8LoadArgs& a, cudaStream_t s);

// A token's slots inv[t * top_k + k] in [0, M): combined into out, or dout
// spread over them (dy, dweights each where given).
struct SlotsArgs {
    const void* y; const void* dout;
    const int32_t* inv; const float* weights;    // weights NULL: 1
    void* out; void* dy; float* dweights;
    uint32_t* err;
    int T, top_k, M, H, dtype, out_dtype;
};
cudaError_t launch_slots_combine(const SlotsArgs& a, cudaStream_t s);
cudaError_t launch_slots_spread(const SlotsArgs& a, cudaStream_t s);

struct NormArgs {
    const void* f; const void* resid;            // f NULL: no branch
    const float* w_post; const float* w_pre; const float* gate;      // each NULL: ones
    void* resid_out; void* x; float* rstd;       // each where given
    int T, H, dtype, resid_dtype, post;
    float alpha, beta, eps;
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s);
// CTAs whose partial weight gradients ([2][H] fp32 each) the workspace holds,
// behind its first kGroupedWsBytes.
constexpr int kNormParts = 608;
struct NormBwdArgs {
    const void* dx; const void* dresid_out;      // each NULL: zeros
    const void* f; const void* resid_out;
    const float* w_post; const float* w_pre; const float* gate; const float* rstd;
    void* df; void* dresid; float* dgate; float* dw_post; float* dw_pre;
    float* parts;
    int T, H, dtype, resid_dtype, post;
    float alpha, beta;
};
cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s);

}  // namespace strata
