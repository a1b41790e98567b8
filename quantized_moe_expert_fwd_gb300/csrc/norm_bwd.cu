// norm_bwd.cu -- the norms around a block, backward (the formulas are in
// norm.cuh).
//
// A row's three sums come from one pass over it, as s0 and s1 are known:
//   m = sum dx wpre r',   A = sum (dr' + s1 dx wpre) wpost f,   B = sum r' wpost f
// give c = s1^3 m / H and sum D wpost f = A - c B.  The weights' gradients are
// summed in the threads' registers over the rows of a CTA, set aside in shared
// memory every kNbPiece rows (equal terms round one way within a binade), and
// the CTAs' sums joined in their order by a second kernel.
#include "norm.cuh"

namespace strata {

namespace {

constexpr int kNbPiece = 256;

template <typename T, typename TR, int C>
struct NormIn {                              // what a thread reads of a row
    Raw<T, 8> dx[C], f[C];
    Raw<TR, 8> v[C], dr2[C];
    float s0, s1, g;
};

template <typename T, typename TR, int W, int C, bool VEC>
__global__ void __launch_bounds__(NormRow<W, C, VEC>::kBlock, W <= 8 ? 2 : 1) k_norm_bwd(NormBwdArgs a, bool wide) {
    using R = NormRow<W, C, VEC>;
    using In = NormIn<T, TR, C>;
    constexpr bool AHEAD = C == 1;           // the next row's loads under way, the weights in registers
    __shared__ float buf[2][R::kGroups][W][3];
    extern __shared__ float aside[];         // [2 C][8][thread]
    const R row;
    pdl_launch();
    pdl_wait();
    const int H = a.H;
    const float inv = 1.0f / float(H);
    const size_t step = size_t(gridDim.x) * R::kGroups;
    auto read = [&](In& in, size_t t) {
        if (t >= size_t(a.T)) return;
        const size_t at = t * H;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.dx) {
                in.dx[c] = row.template load<true>(static_cast<const T*>(a.dx) + at, c, H, false);
                in.v[c] = row.template load<true>(static_cast<const TR*>(a.resid_out) + at, c, H, wide);
            }
            // dr may take its place
            if (a.dresid_out) in.dr2[c] = row.template load<false>(static_cast<const TR*>(a.dresid_out) + at, c, H, wide);
            if (a.f) in.f[c] = row.template load<true>(static_cast<const T*>(a.f) + at, c, H, false);
        }
        in.s0 = __ldg(a.rstd + 2 * t);
        in.s1 = __ldg(a.rstd + 2 * t + 1);
        in.g = a.beta * (a.gate ? __ldg(a.gate + t) : 1.0f);
    };
    auto weight = [&](const float* w, int c, float (&o)[8]) {
        Raw<float, 8> r{};
        if (w) r = row.template load<true>(w, c, H, wide);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = w ? r.get(j) : 1.0f;
    };
    float w_pre[8], w_post[8];
    if (AHEAD) {
        weight(a.w_pre, 0, w_pre);
        weight(a.w_post, 0, w_post);
    }
    float d_pre[C][8] = {}, d_post[C][8] = {};
    int rows = 0;
    bool set = false;
    auto put_aside = [&]() {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float* p = aside + (2 * c * 8 + j) * R::kBlock + threadIdx.x;
                float* q = p + 8 * R::kBlock;
                *p = set ? *p + d_pre[c][j] : d_pre[c][j];
                *q = set ? *q + d_post[c][j] : d_post[c][j];
                d_pre[c][j] = d_post[c][j] = 0.0f;
            }
        set = true;
    };
    In in{};
    size_t t = size_t(blockIdx.x) * R::kGroups + row.group;
    read(in, t);
    for (int n = 0; t < size_t(a.T); t += step, n ^= 1) {
        In next{};
        if (AHEAD) read(next, t + step);
        const size_t at = t * H;
        float q[3] = {};
        float c1 = 0.0f, c0 = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!AHEAD) {
                weight(a.w_pre, c, w_pre);
                weight(a.w_post, c, w_post);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gx = in.dx[c].get(j) * w_pre[j], v = in.v[c].get(j);
                const float wf = w_post[j] * in.f[c].get(j);
                q[0] = fmaf(gx, v, q[0]);
                q[1] = fmaf(fmaf(in.s1, gx, in.dr2[c].get(j)), wf, q[1]);
                q[2] = fmaf(v, wf, q[2]);
            }
        }
        row.sum(q, &buf[n]);
        c1 = in.s1 * in.s1 * in.s1 * (q[0] * inv);
        const float df = q[1] - c1 * q[2];
        if (a.dgate && row.id == 0) a.dgate[t] = a.beta * in.s0 * df;
        if (a.post) c0 = in.g * in.s0 * in.s0 * in.s0 * (df * inv);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!AHEAD) {
                weight(a.w_pre, c, w_pre);
                weight(a.w_post, c, w_post);
            }
            float o[8], r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float dx = in.dx[c].get(j), v = in.v[c].get(j), f = in.f[c].get(j);
                const float d = in.dr2[c].get(j) + fmaf(in.s1, dx * w_pre[j], -c1 * v);
                const float dn = in.g * d;
                d_pre[c][j] = fmaf(dx * v, in.s1, d_pre[c][j]);
                d_post[c][j] = fmaf(dn * f, in.s0, d_post[c][j]);
                o[j] = a.post ? fmaf(in.s0, dn * w_post[j], -c0 * f) : dn;
                r[j] = a.alpha * d;
            }
            if (a.df) row.store(static_cast<T*>(a.df) + at, c, H, o, false);
            if (a.dresid) row.store(static_cast<TR*>(a.dresid) + at, c, H, r, wide);
        }
        if (++rows % kNbPiece == 0) put_aside();
        if (AHEAD) in = next;
        else read(in, t + step);
    }
    if (!a.dw_pre && !a.dw_post) return;
    put_aside();
    __syncthreads();
    // the groups of the block in their order
    float* part = a.parts + size_t(blockIdx.x) * 2 * H;
    if (row.group == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[j] = 0.0f;
                    for (int g = 0; g < R::kGroups; ++g)
                        o[j] += aside[((2 * c + k) * 8 + j) * R::kBlock + g * R::kThreads + row.id];
                }
                if (k == 0 ? a.dw_pre != nullptr : a.dw_post != nullptr)
                    row.store(part + k * H, c, H, o, false);
            }
    }
}

constexpr int kNmRows = 8;               // rows whose weight gradients are added before they meet the others

// Rows of any length.  A CTA takes kNmRows rows at a time: their sums, then column by
// column the gradients and the rows' part of the weights', which is added to
// the CTA's own sums in the workspace ([CTA][2][H]).
template <typename T, typename TR>
__global__ void __launch_bounds__(kNmThreads) k_norm_bwd_any(NormBwdArgs a) {
    __shared__ float buf[kNmThreads / 32];
    __shared__ float c1s[kNmRows], c0s[kNmRows];
    const int H = a.H;
    pdl_launch();
    pdl_wait();
    const float inv = 1.0f / float(H);
    float* part_pre = a.parts + size_t(blockIdx.x) * 2 * H;
    float* part_post = part_pre + H;
    const T* dx = static_cast<const T*>(a.dx);
    const TR* v = static_cast<const TR*>(a.resid_out);
    const TR* dr2 = static_cast<const TR*>(a.dresid_out);
    const T* f = static_cast<const T*>(a.f);
    bool first = true;
    for (size_t t0 = size_t(blockIdx.x) * kNmRows; t0 < size_t(a.T); t0 += size_t(gridDim.x) * kNmRows) {
        const int rows = int(min(size_t(kNmRows), size_t(a.T) - t0));
        // D of one element; c1 = s1^3 mean(dx wpre r')
        auto grad = [&](size_t at, int c, float s1, float c1) {
            float d = dr2 ? to_f32(dr2[at]) : 0.0f;
            if (dx) d += fmaf(s1, to_f32(dx[at]) * (a.w_pre ? a.w_pre[c] : 1.0f), -c1 * to_f32(v[at]));
            return d;
        };
        __syncthreads();
        for (int i = 0; i < rows; ++i) {
            const size_t t = t0 + i, row = t * H;
            const float s0 = a.rstd[2 * t], s1 = a.rstd[2 * t + 1];
            float c1 = 0.0f, c0 = 0.0f;
            if (dx) {
                const float q = cta_sum(column_sum(H, [&](int c) {
                    return to_f32(dx[row + c]) * (a.w_pre ? a.w_pre[c] : 1.0f) * to_f32(v[row + c]);
                }), buf);
                c1 = s1 * s1 * s1 * (q * inv);
            }
            if (a.post || a.dgate) {
                const float q = cta_sum(column_sum(H, [&](int c) {
                    return grad(row + c, c, s1, c1) * (a.w_post ? a.w_post[c] : 1.0f) * to_f32(f[row + c]);
                }), buf);
                if (a.dgate && threadIdx.x == 0) a.dgate[t] = a.beta * s0 * q;
                if (a.post) c0 = a.beta * (a.gate ? a.gate[t] : 1.0f) * s0 * s0 * s0 * (q * inv);
            }
            if (threadIdx.x == 0) {
                c1s[i] = c1;
                c0s[i] = c0;
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < H; c += kNmThreads) {
            float dw_pre = 0.0f, dw_post = 0.0f;
            for (int i = 0; i < rows; ++i) {
                const size_t t = t0 + i, at = t * H + c;
                const float s0 = a.rstd[2 * t], s1 = a.rstd[2 * t + 1];
                const float d = grad(at, c, s1, c1s[i]);
                const float dn = a.beta * (a.gate ? a.gate[t] : 1.0f) * d;
                if (a.dw_pre) dw_pre += to_f32(dx[at]) * to_f32(v[at]) * s1;
                if (a.dw_post) dw_post += dn * to_f32(f[at]) * s0;
                if (a.df) {
                    float o = dn;
                    if (a.post) o = fmaf(s0, dn * (a.w_post ? a.w_post[c] : 1.0f), -c0s[i] * to_f32(f[at]));
                    static_cast<T*>(a.df)[at] = from_f32<T>(o);
                }
                if (a.dresid) static_cast<TR*>(a.dresid)[at] = from_f32<TR>(a.alpha * d);
            }
            if (a.dw_pre) part_pre[c] = first ? dw_pre : part_pre[c] + dw_pre;
            if (a.dw_post) part_post[c] = first ? dw_post : part_post[c] + dw_post;
        }
        first = false;
    }
}

// The CTAs' sums of a column: kJoinRows runs of them, then the runs, in order.
constexpr int kJoinCols = 32, kJoinRows = 8;
__global__ void __launch_bounds__(kJoinCols * kJoinRows) k_norm_join(const float* parts, int n, int H, float* dw_pre,
                                                                     float* dw_post) {
    __shared__ float run[kJoinRows][kJoinCols];
    pdl_launch();
    pdl_wait();
    const int x = threadIdx.x % kJoinCols, y = threadIdx.x / kJoinCols;
    const int c = int(blockIdx.x) * kJoinCols + x;
    const int per = (n + kJoinRows - 1) / kJoinRows;
    float* out = c < H ? dw_pre : dw_post;
    float sum = 0.0f;
    if (c < 2 * H && out != nullptr) {
        const int last = min(n, (y + 1) * per);
#pragma unroll 8
        for (int i = y * per; i < last; ++i) sum += __ldcg(parts + size_t(i) * 2 * H + c);
    }
    run[y][x] = sum;
    __syncthreads();
    if (y != 0 || c >= 2 * H || out == nullptr) return;
    for (int i = 1; i < kJoinRows; ++i) sum += run[i][x];
    out[c < H ? c : c - H] = sum;
}

template <typename T, typename TR, int W, int C, bool VEC>
cudaError_t run_rows(const NormBwdArgs& a, int* n, cudaStream_t s) {
    using R = NormRow<W, C, VEC>;
    const int want = (a.T + R::kGroups - 1) / R::kGroups, most = device_info().sms * (W <= 8 ? 2 : 1);
    *n = want < most ? want : most;
    if (*n > kNormParts) *n = kNormParts;
    if (*n == 0) return cudaSuccess;
    const size_t pitch = size_t(a.H) * sizeof(TR);
    const bool wide = aligned32(a.resid_out, pitch) && aligned32(a.dresid_out, pitch) && aligned32(a.dresid, pitch) &&
                      aligned32(a.w_post, 0) && aligned32(a.w_pre, size_t(a.H) * 4);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(*n);
    cfg.blockDim = dim3(R::kBlock);
    cfg.dynamicSmemBytes = size_t(16) * C * R::kBlock * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_norm_bwd<T, TR, W, C, VEC>, a, wide);
}
template <typename T, typename TR, bool VEC>
cudaError_t run_norm_bwd(const NormBwdArgs& a, int* n, cudaStream_t s) {
    if (a.H <= 256) return run_rows<T, TR, 1, 1, VEC>(a, n, s);
    if (a.H <= 512) return run_rows<T, TR, 2, 1, VEC>(a, n, s);
    if (a.H <= 1024) return run_rows<T, TR, 4, 1, VEC>(a, n, s);
    if (a.H <= 2048) return run_rows<T, TR, 8, 1, VEC>(a, n, s);
    if (a.H <= 4096) return run_rows<T, TR, 16, 1, VEC>(a, n, s);
    const int want = (a.T + kNmRows - 1) / kNmRows;
    *n = want < kNormParts ? want : kNormParts;
    return *n == 0 ? cudaSuccess : row_launch(k_norm_bwd_any<T, TR>, dim3(*n), dim3(kNmThreads), s, a);
}
template <typename T, typename TR>
cudaError_t pick_norm_bwd(const NormBwdArgs& a, int* n, cudaStream_t s) {
    return a.H % 8 == 0 ? run_norm_bwd<T, TR, true>(a, n, s) : run_norm_bwd<T, TR, false>(a, n, s);
}

}  // namespace

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
    int n = 0;
    cudaError_t e;
    if (a.dtype == STRATA_BF16)
        e = a.resid_dtype == STRATA_F32 ? pick_norm_bwd<__nv_bfloat16, float>(a, &n, s)
                                        : pick_norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, &n, s);
    else
        e = a.resid_dtype == STRATA_F32 ? pick_norm_bwd<__half, float>(a, &n, s)
                                        : pick_norm_bwd<__half, __half>(a, &n, s);
    if (e != cudaSuccess || (!a.dw_pre && !a.dw_post)) return e;
    return row_launch(k_norm_join, dim3((2 * a.H + kJoinCols - 1) / kJoinCols), dim3(kJoinCols * kJoinRows), s,
                      static_cast<const float*>(a.parts), n, a.H, a.dw_pre, a.dw_post);
}

}  // namespace strata
