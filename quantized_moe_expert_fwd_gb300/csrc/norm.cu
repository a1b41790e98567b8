// norm.cu -- the norms around a block, forward (the formulas are in norm.cuh).
#include "norm.cuh"

namespace strata {

namespace {

template <typename T, typename TR, int W, int C, bool VEC>
__global__ void __launch_bounds__(NormRow<W, C, VEC>::kBlock) k_norm(NormArgs a) {
    using R = NormRow<W, C, VEC>;
    __shared__ NormSums<1> buf[2][R::kGroups][W];
    const R row;
    pdl_launch();
    pdl_wait();
    const size_t t = size_t(blockIdx.x) * R::kGroups + row.group;
    if (t >= size_t(a.T)) return;
    const int H = a.H;
    const size_t at = t * H;
    Raw<T, 8> rf[C];
    Raw<TR, 8> rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (a.f) rf[c] = row.template load<true>(static_cast<const T*>(a.f) + at, c, H);
        // r' may take r's place
        rr[c] = row.template load<false>(static_cast<const TR*>(a.resid) + at, c, H);
    }
    Raw<float, 8> wpost[VEC ? C : 1];
#pragma unroll
    for (int c = 0; VEC && c < C; ++c)
        if (a.w_post) wpost[c] = row.template load<true>(a.w_post, c, H);
    const float g = a.beta * (a.gate ? __ldg(a.gate + t) : 1.0f);
    const float inv = 1.0f / float(H);
    float s0 = 1.0f, s1 = 1.0f;
    if (a.post) {
        float q[1] = {};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) q[0] = fmaf(rf[c].get(j), rf[c].get(j), q[0]);
        row.sum(q, &buf[0]);
        s0 = 1.0f / sqrtf(q[0] * inv + a.eps);
    }
    float v[C][8];
    float q[1] = {};
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = a.alpha * rr[c].get(j);
        if (a.f) {
            Raw<float, 8> w{};
            if (VEC) w = wpost[VEC ? c : 0];
            else if (a.w_post) w = row.template load<true>(a.w_post, c, H);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float n = rf[c].get(j) * s0;
                if (a.w_post) n *= w.get(j);
                v[c][j] = fmaf(g, n, v[c][j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // as it is stored
            v[c][j] = to_f32(from_f32<TR>(v[c][j]));
            q[0] = fmaf(v[c][j], v[c][j], q[0]);
        }
        if (a.resid_out) row.store(static_cast<TR*>(a.resid_out) + at, c, H, v[c]);
    }
    if (a.x) {
        row.sum(q, &buf[1]);
        s1 = 1.0f / sqrtf(q[0] * inv + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Raw<float, 8> w{};
            if (a.w_pre) w = row.template load<true>(a.w_pre, c, H);
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = a.w_pre ? v[c][j] * s1 * w.get(j) : v[c][j] * s1;
            row.store(static_cast<T*>(a.x) + at, c, H, o);
        }
    }
    if (a.rstd && row.id == 0) {
        a.rstd[2 * t] = s0;
        a.rstd[2 * t + 1] = s1;
    }
}

// Rows of any length: three passes over the row.
template <typename T, typename TR>
__global__ void __launch_bounds__(kNmThreads) k_norm_any(NormArgs a) {
    __shared__ float buf[kNmThreads / 32];
    const int H = a.H;
    pdl_launch();
    pdl_wait();
    for (size_t t = blockIdx.x; t < size_t(a.T); t += gridDim.x) {
        const T* f = static_cast<const T*>(a.f) + t * H;
        const TR* r = static_cast<const TR*>(a.resid) + t * H;
        float s0 = 1.0f;
        if (a.post) {
            const float q = cta_sum(column_sum(H, [&](int c) {
                const float v = to_f32(f[c]);
                return v * v;
            }), buf);
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
            const float q = cta_sum(column_sum(H, [&](int c) {
                const float v = to_f32(stored(c));
                return v * v;
            }), buf);
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

template <typename T, typename TR, int W, int C, bool VEC>
cudaError_t run_rows(const NormArgs& a, cudaStream_t s) {
    using R = NormRow<W, C, VEC>;
    return row_launch(k_norm<T, TR, W, C, VEC>, dim3((a.T + R::kGroups - 1) / R::kGroups), dim3(R::kBlock), s, a);
}

// Sixteen columns a thread (us, 32768 rows of 512 columns, 16384 of 2048, 8192 of
// 4096; at the copy's rate 30, 59, 59): 8 a thread 36.9, 71.2, 66.3; 16 32.5,
// 61.0, 60.9; 32 32.4, 63.2, 63.7; 16 and the weights read with the row 31.1,
// 59.3, 59.3 (columns one by one, 16384 x 1031: 54.8, with them 62.0).
template <typename T, typename TR, bool VEC>
cudaError_t run_norm(const NormArgs& a, cudaStream_t s) {
    if (a.H <= 256) return run_rows<T, TR, 1, 1, VEC>(a, s);
    if (a.H <= 512) return run_rows<T, TR, 1, 2, VEC>(a, s);
    if (a.H <= 1024) return run_rows<T, TR, 2, 2, VEC>(a, s);
    if (a.H <= 2048) return run_rows<T, TR, 4, 2, VEC>(a, s);
    if (a.H <= 4096) return run_rows<T, TR, 8, 2, VEC>(a, s);
    if (a.H <= 8192) return run_rows<T, TR, 16, 2, VEC>(a, s);
    if (a.H <= 16384) return run_rows<T, TR, 32, 2, VEC>(a, s);
    // (2048 rows of 16384 columns: 78 us above, 213 here; of 16383 114 and 220)
    const int most = device_info().sms * 8;
    return row_launch(k_norm_any<T, TR>, dim3(a.T < most ? a.T : most), dim3(kNmThreads), s, a);
}
template <typename T, typename TR>
cudaError_t pick_norm(const NormArgs& a, cudaStream_t s) {
    return a.H % 4 == 0 ? run_norm<T, TR, true>(a, s) : run_norm<T, TR, false>(a, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
    if (a.dtype == STRATA_BF16)
        return a.resid_dtype == STRATA_F32 ? pick_norm<__nv_bfloat16, float>(a, s)
                                           : pick_norm<__nv_bfloat16, __nv_bfloat16>(a, s);
    return a.resid_dtype == STRATA_F32 ? pick_norm<__half, float>(a, s) : pick_norm<__half, __half>(a, s);
}

}  // namespace strata
