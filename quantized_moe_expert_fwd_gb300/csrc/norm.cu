// norm.cu -- the RMS norms before and after a block, its gate and the scales
// of residual and branch, forward and backward.
//   n  = f s0 wpost          s0 = 1 / sqrt(mean f^2 + eps)   (or n = f)
//   r' = alpha r + beta gate n
//   x  = r' s1 wpre          s1 = 1 / sqrt(mean r'^2 + eps)
// Backward, from dx and the gradient dr' of r' by other paths, with
// D = dr' + s1 (dx wpre - r' s1^2 mean(dx wpre r')) the whole gradient by r':
//   dr = alpha D,  dgate = beta sum(D n),  dn = beta gate D
//   df = s0 (dn wpost - f s0^2 mean(dn wpost f))             (or df = dn)
//   dwpre = sum over the rows of dx r' s1,  dwpost = sum of dn f s0
// x is of r' as it is stored, so that the backward pass sees what the forward
// pass did.
#include "grouped.cuh"
#include "grouped.h"

namespace strata {

namespace {

constexpr int kNmThreads = 256;
constexpr int kNmRows = 8;               // rows whose weight gradients are added before they meet the others

// The sum over a CTA, in all its threads; buf: a float a warp, free again
// after the next barrier.
__device__ __forceinline__ float cta_sum(float v, float* buf) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < int(blockDim.x) >> 5; ++i) s += buf[i];
    return s;
}

// A thread's sum of f(c) over its columns of a row, in pieces of 64.
template <typename F>
__device__ __forceinline__ float column_sum(int H, F f) {
    float sum = 0.0f;
    for (int c0 = threadIdx.x; c0 < H; c0 += 64 * kNmThreads) {
        float part = 0.0f;
        for (int c = c0; c < min(H, c0 + 64 * kNmThreads); c += kNmThreads) part += f(c);
        sum += part;
    }
    return sum;
}

// Any width: three passes over the row.
template <typename T, typename TR>
__global__ void __launch_bounds__(kNmThreads) k_norm(NormArgs a) {
    __shared__ float buf[kNmThreads / 32];
    const int H = a.H;
    for (size_t t = blockIdx.x; t < size_t(a.T); t += gridDim.x) {
        const T* f = static_cast<const T*>(a.f) + t * H;
        const TR* r = static_cast<const TR*>(a.resid) + t * H;
        float s0 = 1.0f;
        if (a.post) {
            const float q = cta_sum(column_sum(H, [&](int c) { const float v = to_f32(f[c]); return v * v; }), buf);
            s0 = 1.0f / sqrtf(q / float(H) + a.eps);
        }
        const float g = a.beta * (a.gate ? a.gate[t] : 1.0f);
        auto stored = [&](int c) {
            float v = a.alpha * to_f32(r[c]);
            if (a.f) {
                float n = to_f32(f[c]) * s0;
                if (a.w_post) n *= a.w_post[c];
                v = fmaf(g, n, v);
            }
            return from_f32<TR>(v);
        };
        float s1 = 1.0f;
        if (a.x) {
            const float q = cta_sum(column_sum(H, [&](int c) { const float v = to_f32(stored(c)); return v * v; }), buf);
            s1 = 1.0f / sqrtf(q / float(H) + a.eps);
        }
        // r' may take r's place: a column is read once more and then written, by one thread
        for (int c = threadIdx.x; c < H; c += kNmThreads) {
            const TR v = stored(c);
            if (a.x) {
                const float n = to_f32(v) * s1;
                static_cast<T*>(a.x)[t * H + c] = from_f32<T>(a.w_pre ? n * a.w_pre[c] : n);
            }
            if (a.resid_out) static_cast<TR*>(a.resid_out)[t * H + c] = v;
        }
        if (a.rstd && threadIdx.x == 0) {
            a.rstd[2 * t] = s0;
            a.rstd[2 * t + 1] = s1;
        }
    }
}

// Any width.  A CTA takes kNmRows rows at a time: their sums, then column by
// column the gradients and the rows' part of the weights', which is added to
// the CTA's own sums in the workspace ([CTA][2][H]).
template <typename T, typename TR>
__global__ void __launch_bounds__(kNmThreads) k_norm_bwd(NormBwdArgs a) {
    __shared__ float buf[kNmThreads / 32];
    __shared__ float c1s[kNmRows], c0s[kNmRows];
    const int H = a.H;
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

// The CTAs' sums of a column, in their order.
__global__ void __launch_bounds__(kNmThreads) k_norm_join(const float* parts, int n, int H, float* dw_pre,
                                                          float* dw_post) {
    const int c = int(blockIdx.x) * kNmThreads + int(threadIdx.x);
    if (c >= 2 * H) return;
    float* out = c < H ? dw_pre : dw_post;
    if (out == nullptr) return;
    float sum = 0.0f;
    for (int i = 0; i < n; ++i) sum += parts[size_t(i) * 2 * H + c];
    out[c < H ? c : c - H] = sum;
}

template <typename T, typename TR>
cudaError_t run_norm(const NormArgs& a, cudaStream_t s) {
    const int most = device_info().sms * 8;
    k_norm<T, TR><<<a.T < most ? a.T : most, kNmThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, typename TR>
cudaError_t run_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
    const int want = (a.T + kNmRows - 1) / kNmRows, n = want < kNormParts ? want : kNormParts;
    if (n > 0) {
        k_norm_bwd<T, TR><<<n, kNmThreads, 0, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.dw_pre || a.dw_post)
        k_norm_join<<<(2 * a.H + kNmThreads - 1) / kNmThreads, kNmThreads, 0, s>>>(a.parts, n, a.H, a.dw_pre,
                                                                                   a.dw_post);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
    if (a.dtype == STRATA_BF16)
        return a.resid_dtype == STRATA_F32 ? run_norm<__nv_bfloat16, float>(a, s)
                                           : run_norm<__nv_bfloat16, __nv_bfloat16>(a, s);
    return a.resid_dtype == STRATA_F32 ? run_norm<__half, float>(a, s) : run_norm<__half, __half>(a, s);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
    if (a.dtype == STRATA_BF16)
        return a.resid_dtype == STRATA_F32 ? run_norm_bwd<__nv_bfloat16, float>(a, s)
                                           : run_norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, s);
    return a.resid_dtype == STRATA_F32 ? run_norm_bwd<__half, float>(a, s)
                                       : run_norm_bwd<__half, __half>(a, s);
}

}  // namespace strata
