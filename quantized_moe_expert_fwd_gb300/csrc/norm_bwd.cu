// norm_bwd.cu -- the norms around a block, backward (the formulas are in
// norm.cuh).
//
// A row's three sums come from one pass over it, as s0 and s1 are known:
//   m = sum dx wpre r',   A = sum (dr' + s1 dx wpre) wpost f,   B = sum r' wpost f
// give D = dr' + s1 dx wpre - e (s1 r') and sum D wpost f = A - e (s1 B) with
// e = s1 (s1 m / H).  The factors are multiplied so that none leaves fp32 before
// the gradient does: s1^3 would for rows of root mean square 1e13 (its digits go;
// at 1e15 the whole term) or, where eps lets them be, 1e-13 (infinite).
//
// The weights' gradients are summed in the threads' registers over the rows of a
// CTA, set aside every kNbPiece rows (equal terms round one way within a binade;
// in shared memory, or where a CTA has one row at a time in its own part of the
// workspace), and the CTAs' sums joined in their order by a second kernel.
//
// 16384 rows of 2048 columns (bf16, fp32 residual; us; at the copy's rate 89, and
// about 4 for the join), as it was built: rows read once a pass 420; in
// registers, the next row's loads under way 129; 8 neighbouring columns a lane
// copied ahead (16-byte copies then fetch fp32's sectors twice) 130 with 2, 3
// or 4 rows; fours of columns 118; packed fp32 117; two rows a step under one
// barrier 99.  Three CTAs an SM (85 registers) spill: 300.  Sixteen columns a
// thread instead of two rows: 139.
#include "grouped_tc.cuh"
#include "norm.cuh"

namespace strata {

namespace {

constexpr int kNbPiece = 256;                  // rows

// Two columns at once (packed fp32).
__device__ __forceinline__ uint64_t both(float v) { return pk(v, v); }
__device__ __forceinline__ float halves(uint64_t v) {
    const float2 f = upk(v);
    return f.x + f.y;
}
template <typename T>
__device__ __forceinline__ uint64_t pair(const Raw<T, 8>& r, int i) { return pk(r.get(2 * i), r.get(2 * i + 1)); }

template <typename T>
__device__ __forceinline__ void clear(Raw<T, 8>& r, int j) {
    if constexpr (sizeof(T) == 4) r.w[j] = 0;
    else r.w[j >> 1] &= j & 1 ? 0xffffu : 0xffff0000u;
}

template <typename T, typename TR>
struct NormCols {                            // eight columns of a row
    Raw<T, 8> dx, f;
    Raw<TR, 8> v, dr2;
};
struct NormScalars {
    float s0, s1, gate;
};

// Rows on their way: each thread copies its own columns of the next rows to its
// own places in shared memory (fours of columns, no barrier), and reads them
// there when their turn comes; what does not exist is filled with zeros.
// kNbSteps steps of ROWS rows.
constexpr int kNbSteps = 2;
template <typename T, typename TR, int W, int C, int ROWS>
struct NormRing {
    static constexpr int kBlock = NormRow<W, C, true>::kBlock;
    static constexpr uint32_t kT = uint32_t(kBlock) * 4 * sizeof(T), kTR = uint32_t(kBlock) * 4 * sizeof(TR);
    static constexpr uint32_t kChunk = 4 * kT + 4 * kTR;     // dx, f; r', dr': twice four columns
    static constexpr uint32_t kBytes = kNbSteps * ROWS * C * kChunk;
    uint8_t* base;
    // Piece k (0 dx, 1 f, 2 r', 3 dr') of chunk c, half h; slot: a row's place.
    template <typename E>
    __device__ __forceinline__ uint8_t* at(int slot, int c, int k, int h) const {
        return base + (slot * C + c) * kChunk +
               (k < 2 ? (2 * k + h) * kT : 4 * kT + (2 * (k - 2) + h) * kTR) + threadIdx.x * (4 * sizeof(E));
    }
    // n of four elements from src + from on.
    template <typename E>
    __device__ __forceinline__ void copy(const E* src, size_t from, int n, int slot, int c, int k, int h) const {
        const uint32_t dst = smem_u32(at<E>(slot, c, k, h));
        const uint32_t bytes = src != nullptr ? n * sizeof(E) : 0;
        if (bytes) src += from;
        if constexpr (sizeof(E) == 4)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                         : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                         : "memory");
    }
    template <typename E>
    __device__ __forceinline__ void take(Raw<E, 8>& r, int slot, int c, int k) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (sizeof(E) == 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(at<E>(slot, c, k, h));
                r.w[4 * h] = v.x; r.w[4 * h + 1] = v.y; r.w[4 * h + 2] = v.z; r.w[4 * h + 3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(at<E>(slot, c, k, h));
                r.w[2 * h] = v.x; r.w[2 * h + 1] = v.y;
            }
        }
    }
};

// Where the weights' gradients are put aside: a block of one row at a time keeps
// them in its own part of the workspace, others in shared memory, [row of the
// block][2][columns].
template <typename R, int C>
constexpr uint32_t kNbAside = R::kGroups == 1 ? 0 : 16 * C * R::kBlock * sizeof(float);

// ROWS rows a step share a barrier, and hide each other's latencies (a row of one
// warp has no barrier: two a step only cost registers, 65536 x 256 52 us with
// one, 62 with two; 131072 x 64 67 and 85).  VEC: rows
// of whole fours.  Others start and end within one; the copies take those
// fours whole, and the columns of the rows beside are set to zero where a warp
// has such (one column an access instead: 16384 x 1031 138 us, now 89; 8192 x
// 2045 85, 60; 6000 x 3999 141, 88; at the copy's rate 45, 44, 64).
template <typename T, typename TR, int W, int C, bool VEC, int ROWS>
__global__ void __launch_bounds__(NormRow<W, C, true>::kBlock, W <= 8 ? 2 : 1) k_norm_bwd(NormBwdArgs a) {
    using R = NormRow<W, C, true>;
    using Ring = NormRing<T, TR, W, C, ROWS>;
    using Cols = NormCols<T, TR>;
    constexpr bool KEEP = C == 1;            // the norms' weights in registers
    __shared__ NormSums<3 * ROWS> buf[2][R::kGroups][W];
    extern __shared__ __align__(16) uint8_t nb_dyn[];
    const Ring ring{nb_dyn + kNbAside<R, C>};
    const R row;
    pdl_launch();
    pdl_wait();
    const int H = a.H;
    const float inv = 1.0f / float(H);
    const size_t step = size_t(gridDim.x) * R::kGroups, total = size_t(a.T) * H;
    const T* pdx = static_cast<const T*>(a.dx);
    const T* pf = static_cast<const T*>(a.f);
    const TR* pv = a.dx ? static_cast<const TR*>(a.resid_out) : nullptr;
    const TR* pr = static_cast<const TR*>(a.dresid_out);
    size_t t = size_t(blockIdx.x) * R::kGroups + row.group;
    // columns of a row's first four that belong to the row before: the same for all
    // of a thread's rows, as the grid is a whole number of fours of rows
    const int off = VEC ? 0 : int((t * H) & 3);
    auto column = [&](int c, int h) { return row.column(c, 4 * h) - off; };
    auto live = [&](int col) { return col >= 0 && col < H; };
    bool ends = false;                       // whether a four of the warp reaches past its row
    if (!VEC) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = column(c, h);
                ends |= col < 0 || (col < H && col + 4 > H);
            }
        ends = __any_sync(0xffffffffu, ends);
    }
    // starts the copies of rows t, t + step ..
    auto start = [&](size_t t, int at_step) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = column(c, h), slot = at_step * ROWS + r;
                    const size_t at = (t + r * step) * H + col;
                    int n = t + r * step < size_t(a.T) && col < H ? 4 : 0;
                    if (!VEC && n && total - at < 4) n = int(total - at);     // the tensor's end
                    ring.copy(pdx, at, n, slot, c, 0, h);
                    ring.copy(pf, at, n, slot, c, 1, h);
                    ring.copy(pv, at, n, slot, c, 2, h);
                    ring.copy(pr, at, n, slot, c, 3, h);
                }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto from_ring = [&](int slot, int c) {
        Cols o;
        ring.take(o.dx, slot, c, 0);
        ring.take(o.f, slot, c, 1);
        ring.take(o.v, slot, c, 2);
        ring.take(o.dr2, slot, c, 3);
        if (!VEC && ends) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (!live(column(c, j / 4) + j % 4)) {
                    clear(o.dx, j);
                    clear(o.f, j);
                    clear(o.v, j);
                    clear(o.dr2, j);
                }
        }
        return o;
    };
    auto store = [&](auto* p, int c, const float (&v)[8], bool fours) {
        using E = typename std::remove_pointer<decltype(p)>::type;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int col = column(c, h);
            if (fours) {
                if (col < H) st_row<E, 4>(p + col, reinterpret_cast<const float(&)[4]>(v[4 * h]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (live(col + j)) p[col + j] = from_f32<E>(v[4 * h + j]);
            }
        }
    };
    // eight columns of a vector [H]
    auto values = [&](const float* w, int c) {
        Raw<float, 8> r{};
        if constexpr (VEC) {
            r = row.template load<false>(w, c, H);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = column(c, j / 4) + j % 4;
                if (live(col)) r.w[j] = __float_as_uint(w[col]);
            }
        }
        return r;
    };
    auto weight = [&](const float* w, int c, uint64_t (&o)[4]) {
        Raw<float, 8> r{};
        if (w) r = values(w, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = w ? pair(r, i) : both(1.0f);
    };
    uint64_t w_pre[4], w_post[4];
    if (KEEP) {
        weight(a.w_pre, 0, w_pre);
        weight(a.w_post, 0, w_post);
    }
    uint64_t d_pre[C][4] = {}, d_post[C][4] = {};
    int rows = 0;
    bool set = false;
    float* out = a.parts + size_t(blockIdx.x) * 2 * H;
    auto put_aside = [&]() {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint64_t(&d)[4] = k == 0 ? d_pre[c] : d_post[c];
                float o[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = upk(d[i]);
                    o[2 * i] = v.x;
                    o[2 * i + 1] = v.y;
                    d[i] = 0;
                }
                if (R::kGroups == 1 && (k == 0 ? a.dw_pre == nullptr : a.dw_post == nullptr)) continue;
                float* to = (R::kGroups == 1 ? out : reinterpret_cast<float*>(nb_dyn) + row.group * 2 * H) + k * H;
                if (set) {
                    const Raw<float, 8> had = values(to, c);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] += had.get(j);
                }
                store(to, c, o, VEC);
            }
        set = true;
    };
    // read whether there is such a row, a gate, or not, so that nothing waits
    // for the values before their row's turn
    const float* pgate = a.gate ? a.gate : a.rstd;
    auto scalars = [&](size_t t) {
        t = min(t, size_t(a.T) - 1);
        return NormScalars{__ldg(a.rstd + 2 * t), __ldg(a.rstd + 2 * t + 1), __ldg(pgate + t)};
    };
    NormScalars ahead[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) ahead[r] = scalars(t + r * step);
    start(t, 0);
    for (int n = 0; t < size_t(a.T); t += ROWS * step, n ^= 1) {
        start(t + ROWS * step, n ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        float s0[ROWS], s1[ROWS], g[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const bool there = t + r * step < size_t(a.T);
            s0[r] = there ? ahead[r].s0 : 0.0f;
            s1[r] = there && a.dx ? ahead[r].s1 : 0.0f;      // (infinite times no dx is no number)
            g[r] = !there ? 0.0f : a.gate ? a.beta * ahead[r].gate : a.beta;
            ahead[r] = scalars(t + (ROWS + r) * step);
        }
        // dr' + s1 dx wpre, kept for the second pass
        uint64_t part[ROWS][C][4];
        float q[3 * ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            uint64_t q0 = 0, q1 = 0, q2 = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (!KEEP) {
                    weight(a.w_pre, c, w_pre);
                    weight(a.w_post, c, w_post);
                }
                const Cols in = from_ring(n * ROWS + r, c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t gx = mul2(pair(in.dx, i), w_pre[i]), v = pair(in.v, i);
                    const uint64_t wf = mul2(w_post[i], pair(in.f, i));
                    part[r][c][i] = ffma2(both(s1[r]), gx, pair(in.dr2, i));
                    q0 = ffma2(gx, v, q0);
                    q1 = ffma2(part[r][c][i], wf, q1);
                    q2 = ffma2(v, wf, q2);
                }
            }
            q[3 * r] = halves(q0);
            q[3 * r + 1] = halves(q1);
            q[3 * r + 2] = halves(q2);
        }
        row.sum(q, &buf[n]);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const size_t tr = t + r * step, at = tr * H;
            if (tr >= size_t(a.T)) break;
            const float e = s1[r] * (s1[r] * (q[3 * r] * inv));
            const float dn_f = q[3 * r + 1] - e * (s1[r] * q[3 * r + 2]);    // sum of D wpost f
            if (a.dgate && row.id == 0) a.dgate[tr] = a.beta * (s0[r] * dn_f);
            const float m0 = s0[r] * (s0[r] * (dn_f * inv));
            const uint64_t ne = both(-e), nm0 = both(-m0), gs = both(g[r] * s0[r]);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (!KEEP) weight(a.w_post, c, w_post);
                const Cols in = from_ring(n * ROWS + r, c);
                float o[8], p[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t v = mul2(both(s1[r]), pair(in.v, i)), f = pair(in.f, i);
                    const uint64_t d = ffma2(ne, v, part[r][c][i]);
                    // (with s1 r' from above: 4096 x 8192 150 us, now 145)
                    d_pre[c][i] = ffma2(both(s1[r]), mul2(pair(in.dx, i), pair(in.v, i)), d_pre[c][i]);
                    d_post[c][i] = ffma2(gs, mul2(d, f), d_post[c][i]);
                    const float2 x = upk(mul2(gs, a.post ? ffma2(nm0, f, mul2(d, w_post[i])) : d));
                    const float2 y = upk(mul2(both(a.alpha), d));
                    o[2 * i] = x.x;
                    o[2 * i + 1] = x.y;
                    p[2 * i] = y.x;
                    p[2 * i + 1] = y.y;
                }
                if (a.df) store(static_cast<T*>(a.df) + at, c, o, !ends);
                if (a.dresid) store(static_cast<TR*>(a.dresid) + at, c, p, !ends);
            }
        }
        if (++rows % (kNbPiece / ROWS) == 0) put_aside();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!a.dw_pre && !a.dw_post) return;
    put_aside();
    if constexpr (R::kGroups == 1) return;
    __syncthreads();
    // the groups of the block in their order
    for (int c = int(threadIdx.x); c < 2 * H; c += R::kBlock) {
        if (c < H ? a.dw_pre == nullptr : a.dw_post == nullptr) continue;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < R::kGroups; ++i) sum += reinterpret_cast<const float*>(nb_dyn)[i * 2 * H + c];
        out[c] = sum;
    }
}

constexpr int kNmRows = 8;               // rows whose weight gradients are added before they meet the others

// Rows of any length.  A CTA takes kNmRows rows at a time: their sums, then column by
// column the gradients and the rows' part of the weights', which is added to
// the CTA's own sums in the workspace ([CTA][2][H]).
template <typename T, typename TR>
__global__ void __launch_bounds__(kNmThreads) k_norm_bwd_any(NormBwdArgs a) {
    __shared__ float buf[kNmThreads / 32];
    __shared__ float es[kNmRows], m0s[kNmRows];
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
        // D of one element; e = s1^2 mean(dx wpre r')
        auto grad = [&](size_t at, int c, float s1, float e) {
            float d = dr2 ? to_f32(dr2[at]) : 0.0f;
            if (dx) d += fmaf(s1, to_f32(dx[at]) * (a.w_pre ? a.w_pre[c] : 1.0f), -e * (s1 * to_f32(v[at])));
            return d;
        };
        __syncthreads();
        for (int i = 0; i < rows; ++i) {
            const size_t t = t0 + i, row = t * H;
            const float s0 = a.rstd[2 * t], s1 = a.rstd[2 * t + 1];
            float e = 0.0f, m0 = 0.0f;
            if (dx) {
                const float q = cta_sum(column_sum(H, [&](int c) {
                    return to_f32(dx[row + c]) * (a.w_pre ? a.w_pre[c] : 1.0f) * to_f32(v[row + c]);
                }), buf);
                e = s1 * (s1 * (q * inv));
            }
            if (a.post || a.dgate) {
                const float q = cta_sum(column_sum(H, [&](int c) {
                    return grad(row + c, c, s1, e) * (a.w_post ? a.w_post[c] : 1.0f) * to_f32(f[row + c]);
                }), buf);
                if (a.dgate && threadIdx.x == 0) a.dgate[t] = a.beta * (s0 * q);
                m0 = s0 * (s0 * (q * inv));
            }
            if (threadIdx.x == 0) {
                es[i] = e;
                m0s[i] = m0;
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < H; c += kNmThreads) {
            float dw_pre = 0.0f, dw_post = 0.0f;
            for (int i = 0; i < rows; ++i) {
                const size_t t = t0 + i, at = t * H + c;
                const float s0 = a.rstd[2 * t], s1 = a.rstd[2 * t + 1];
                const float d = grad(at, c, s1, es[i]);
                const float g = a.beta * (a.gate ? a.gate[t] : 1.0f), dn = g * d;
                if (a.dw_pre) dw_pre += to_f32(dx[at]) * to_f32(v[at]) * s1;
                if (a.dw_post) dw_post += dn * to_f32(f[at]) * s0;
                if (a.df) {
                    float o = dn;
                    if (a.post)
                        o = g * s0 * fmaf(-m0s[i], to_f32(f[at]), d * (a.w_post ? a.w_post[c] : 1.0f));
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
__global__ void __launch_bounds__(kJoinCols * kJoinRows)
    k_norm_join(const float* parts, int n, int H, float* dw_pre, float* dw_post) {
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

// (8192 rows of 4096 columns: 16 warps and two rows a step 106 us, one row 142,
// 8 warps of 16 columns a thread 120; 4096 of 8192: 145, read once a pass 390;
// 4096 of 6521, which is no whole number of fours: 175 and 327.  Longer rows,
// from 8190 on where they are no whole fours: read once a pass, 4096 of 8190 400
// us where 8189 take 198, 16 of 8196 150.)
template <typename T, typename TR, int W, int C, bool VEC>
cudaError_t run_rows(const NormBwdArgs& a, int* n, cudaStream_t s) {
    constexpr int ROWS = C == 1 && W > 1 ? 2 : 1;
    using R = NormRow<W, C, true>;
    const int want = (a.T + R::kGroups - 1) / R::kGroups, most = device_info().sms * (W <= 8 ? 2 : 1);
    *n = want < most ? want : most;
    if (*n > kNormParts) *n = kNormParts;
    if (*n == 0) return cudaSuccess;
    // where a thread has several rows: a whole number of fours of rows in the grid
    constexpr int FOURS = R::kGroups >= 4 ? 1 : 4 / R::kGroups;
    if (!VEC && *n < want) *n = *n < FOURS ? FOURS : *n - *n % FOURS;
    const size_t dyn = kNbAside<R, C> + NormRing<T, TR, W, C, ROWS>::kBytes;
    return gt_launch<k_norm_bwd<T, TR, W, C, VEC, ROWS>>(R::kBlock, 1, *n, dyn, s, a);
}
template <typename T, typename TR, bool VEC>
cudaError_t run_norm_bwd(const NormBwdArgs& a, int* n, cudaStream_t s) {
    const int wide = VEC ? a.H : a.H + 3;    // a row that starts within a four has one more
    if (wide <= 256) return run_rows<T, TR, 1, 1, VEC>(a, n, s);
    if (wide <= 512) return run_rows<T, TR, 2, 1, VEC>(a, n, s);
    if (wide <= 1024) return run_rows<T, TR, 4, 1, VEC>(a, n, s);
    if (wide <= 2048) return run_rows<T, TR, 8, 1, VEC>(a, n, s);
    if (wide <= 4096) return run_rows<T, TR, 16, 1, VEC>(a, n, s);
    if (wide <= 8192) return run_rows<T, TR, 16, 2, VEC>(a, n, s);
    const int want = (a.T + kNmRows - 1) / kNmRows;
    *n = want < kNormParts ? want : kNormParts;
    return *n == 0 ? cudaSuccess : row_launch(k_norm_bwd_any<T, TR>, dim3(*n), dim3(kNmThreads), s, a);
}
template <typename T, typename TR>
cudaError_t pick_norm_bwd(const NormBwdArgs& a, int* n, cudaStream_t s) {
    return a.H % 4 == 0 ? run_norm_bwd<T, TR, true>(a, n, s) : run_norm_bwd<T, TR, false>(a, n, s);
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
