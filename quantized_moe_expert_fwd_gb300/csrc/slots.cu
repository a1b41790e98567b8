// slots.cu -- a token's slots weighted into its row, and the gradients of
// that: its row's gradient spread over its slots, the weights' as dot products.
//   combine  out[t] = sum_k w[t][k] y[slot(t, k)]
//   spread   dy[slot(t, k)] = w[t][k] dout[t],  dw[t][k] = <dout[t], y[slot(t, k)]>
// Both are bound by memory: each row of y, dy, dout and out moves once.  A
// thread has V columns of one token (V the most that the rows' alignment lets
// one access take), so a token's row is read and written once however many
// slots it has, and the loads of kSlAhead slots are under way together.
// 2048 tokens of 8 slots, 2048 columns, bf16: combine 14.4 us (5.2 TB/s), spread
// with the weights' gradients 25.6 (5.5); the gather of 16384 tokens into 65536
// slots 51 (6.6).  1031 columns, V = 1: 23 and 34.
#include "grouped.h"
#include "rows.cuh"

namespace strata {

namespace {

// Slots whose loads are under way together, and most threads along a token's
// row (2048 tokens of 8 slots and 2048 columns, spread with weights' gradients;
// 16384 tokens gathered into 65536 slots; us): 256 threads and 8 slots 36, 65;
// 256 and 4 33, 62; 128 and 8 29.5, 55; 128 and 4 28.6, 51 (at the copy's rate
// 21, 49).
constexpr int kSlAhead = 4;
constexpr int kSlThreads = 128;
// Accesses of a row whose products a thread adds before it sets the sum aside:
// within a binade equal terms all round one way, and 8192 one after the other
// came out 1.2e-4 off.  The kernels of longer rows, which have a block each, are
// their own (LONG): the checks cost them up to 8 % (200 tokens of 2 slots, 40001
// columns: 201 us, now 215), and others 4 to 10 % (2048 tokens of 8 slots: 28.2).
constexpr int kSlPiece = 64;

// The slots k0 .. of a token and their weights (-1, 0 where there is none).
// Returns whether one lies outside [0, M).
__device__ __forceinline__ bool slots_of(const SlotsArgs& a, size_t t, int k0, int (&slot)[kSlAhead],
                                         float (&w)[kSlAhead]) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kSlAhead; ++i) {
        const int k = k0 + i;
        slot[i] = -1;
        w[i] = 0.0f;
        if (k >= a.top_k) continue;
        const int s = __ldg(a.inv + t * a.top_k + k);
        w[i] = a.weights ? __ldg(a.weights + t * a.top_k + k) : 1.0f;
        if (s < 0 || s >= a.M) bad = true;
        else slot[i] = s;
    }
    return bad;
}

// Block (bx, by): by tokens, bx threads along a row; grid.y pieces of a row.
template <typename T, typename TO, int V>
__global__ void __launch_bounds__(kSlThreads) k_slots_combine(SlotsArgs a, bool wide_out) {
    pdl_launch();
    pdl_wait();
    const size_t t = size_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const int c = int(blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (t >= size_t(a.T) || c >= a.H) return;
    const T* y = static_cast<const T*>(a.y) + c;
    float sum[V] = {};
    for (int k0 = 0; k0 < a.top_k; k0 += kSlAhead) {
        int slot[kSlAhead];
        float w[kSlAhead];
        const bool bad = slots_of(a, t, k0, slot, w);
        Raw<T, V> r[kSlAhead];
#pragma unroll
        for (int i = 0; i < kSlAhead; ++i)
            if (slot[i] >= 0) r[i] = ld_row<T, V>(y + size_t(slot[i]) * a.H);
#pragma unroll
        for (int i = 0; i < kSlAhead; ++i)
            if (slot[i] >= 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) sum[j] = fmaf(w[i], r[i].get(j), sum[j]);
            }
        if (bad && c == 0) latch(a.err, STRATA_EBADROUTE);
    }
    st_row<TO, V>(static_cast<TO*>(a.out) + t * a.H + c, sum, wide_out);
}

// Block (bx, by) as above, but the threads of a token take its whole row: bx
// up to 32 for several tokens a block, by = 1 above; grid.y pieces of their
// slots.  DW: dweights too.
// (Eight blocks an SM, 64 registers, where an access has eight columns: 25.6 us
// instead of 28.6 above; where it has one: 35 instead of 34.)
template <typename T, int V, bool DW, bool LONG>
__global__ void __launch_bounds__(kSlThreads, V == 8 ? 8 : 0) k_slots_spread(SlotsArgs a) {
    __shared__ float part[kSlThreads / 32][kSlAhead];
    __shared__ float aside[LONG ? kSlAhead : 1][LONG ? kSlThreads : 1];
    pdl_launch();
    pdl_wait();
    const size_t t = size_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = t < size_t(a.T);
    const T* dout = static_cast<const T*>(a.dout) + (live ? t : 0) * a.H;
    const T* y = static_cast<const T*>(a.y);
    T* dy = static_cast<T*>(a.dy);
    const int first = int(threadIdx.x) * V;
    // under way while the slots' numbers come
    Raw<T, V> ahead{};
    if (first < a.H) ahead = ld_row<T, V>(dout + first);
    for (int k0 = int(blockIdx.y) * kSlAhead; k0 < a.top_k; k0 += int(gridDim.y) * kSlAhead) {
        int slot[kSlAhead];
        float w[kSlAhead], dot[kSlAhead] = {};
        const bool bad = slots_of(a, live ? t : 0, k0, slot, w);
        int next = first + kSlPiece * kSlThreads * V;        // the next piece (LONG)
        if (LONG) {
#pragma unroll
            for (int i = 0; i < kSlAhead; ++i) aside[i][threadIdx.x] = 0.0f;
        }
        for (int c = first; live && c < a.H; c += int(blockDim.x) * V) {
            if (LONG && c == next) {
                next += kSlPiece * kSlThreads * V;
#pragma unroll
                for (int i = 0; i < kSlAhead; ++i) {
                    aside[i][threadIdx.x] += dot[i];
                    dot[i] = 0.0f;
                }
            }
            const Raw<T, V> rd = c == first ? ahead : ld_row<T, V>(dout + c);
            Raw<T, V> r[kSlAhead];
            if (DW) {
#pragma unroll
                for (int i = 0; i < kSlAhead; ++i)
                    if (slot[i] >= 0) r[i] = ld_row<T, V>(y + size_t(slot[i]) * a.H + c);
            }
            float d[V];
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = rd.get(j);
#pragma unroll
            for (int i = 0; i < kSlAhead; ++i) {
                if (slot[i] < 0) continue;
                if (dy) {
                    T* p = dy + size_t(slot[i]) * a.H + c;
                    if (a.weights) {
                        float o[V];
#pragma unroll
                        for (int j = 0; j < V; ++j) o[j] = w[i] * d[j];
                        st_row<T, V>(p, o);
                    } else if constexpr (Raw<T, V>::kBytes == 2) {
                        *reinterpret_cast<uint16_t*>(p) = uint16_t(rd.w[0]);
                    } else {
                        st_words(p, false, rd.w);
                    }
                }
                if (DW) {
                    // a row's thread sums V columns at a time
                    float s = 0.0f;
#pragma unroll
                    for (int j = 0; j < V; ++j) s = fmaf(d[j], r[i].get(j), s);
                    dot[i] += s;
                }
            }
        }
        if (bad && live && threadIdx.x == 0) latch(a.err, STRATA_EBADROUTE);
        if (!DW) continue;
#pragma unroll
        for (int i = 0; i < kSlAhead; ++i) {
            if (LONG) dot[i] += aside[i][threadIdx.x];       // its own
            dot[i] = group_sum(dot[i], min(32, int(blockDim.x)));
        }
        float* out = a.dweights + t * a.top_k + k0;
        if (blockDim.x <= 32) {
#pragma unroll
            for (int i = 0; i < kSlAhead; ++i)
                if (live && threadIdx.x == 0 && k0 + i < a.top_k) out[i] = dot[i];
            continue;
        }
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kSlAhead; ++i) part[warp][i] = dot[i];
        }
        __syncthreads();
        if (threadIdx.x < kSlAhead && k0 + int(threadIdx.x) < a.top_k) {
            float s = 0.0f;
            for (int i = 0; i < int(blockDim.x) >> 5; ++i) s += part[i][threadIdx.x];
            out[threadIdx.x] = s;
        }
        __syncthreads();
    }
}

// Threads along a row of `units` accesses: a power of two.
int threads_along(int units, int most) {
    int n = 1;
    while (n < units && n < most) n *= 2;
    return n;
}

template <typename T, typename TO, int V>
cudaError_t run_combine(const SlotsArgs& a, cudaStream_t s) {
    const int units = (a.H + V - 1) / V, bx = threads_along(units, kSlThreads), by = kSlThreads / bx;
    const dim3 grid((a.T + by - 1) / by, (units + bx - 1) / bx);
    return row_launch(k_slots_combine<T, TO, V>, grid, dim3(bx, by), s, a,
                      aligned32(a.out, size_t(a.H) * sizeof(TO)));
}
template <typename T, int V>
cudaError_t run_spread(const SlotsArgs& a, cudaStream_t s) {
    const int units = (a.H + V - 1) / V, bx = threads_along(units, kSlThreads);
    const int by = bx <= 32 ? kSlThreads / bx : 1;
    // Few tokens: their slots in pieces side by side.  (8 slots, 2048 columns, with
    // the weights' gradients, us, side by side and in a row: 16 tokens 3.2 and 5.2,
    // 304 5.0 and 7.7, 608 9.3 and 11.4, 1216 16.3 and 15.8, 2432 30.3 and 28.9; the
    // gather 1.9 and 2.5, 3.6 and 3.8, 5.0 and 6.0, 8.2 and 8.5, 15.4 both, but 456
    // tokens 4.2 and 3.7, of 5 slots 304 3.4 and 2.9, 456 3.8 and 3.0.  Hence two
    // tokens an SM.)
    const int pieces = a.T <= device_info().sms * 2 ? (a.top_k + kSlAhead - 1) / kSlAhead : 1;
    const dim3 grid((a.T + by - 1) / by, pieces);
    if (!a.dweights) return row_launch(k_slots_spread<T, V, false, false>, grid, dim3(bx, by), s, a);
    return a.H > kSlPiece * kSlThreads * V ? row_launch(k_slots_spread<T, V, true, true>, grid, dim3(bx, by), s, a)
                                           : row_launch(k_slots_spread<T, V, true, false>, grid, dim3(bx, by), s, a);
}

template <typename T, typename TO>
cudaError_t pick_combine(const SlotsArgs& a, cudaStream_t s) {
    return a.H % 8 == 0   ? run_combine<T, TO, 8>(a, s)
           : a.H % 4 == 0 ? run_combine<T, TO, 4>(a, s)
           : a.H % 2 == 0 ? run_combine<T, TO, 2>(a, s)
                          : run_combine<T, TO, 1>(a, s);
}
template <typename T>
cudaError_t pick_spread(const SlotsArgs& a, cudaStream_t s) {
    return a.H % 8 == 0   ? run_spread<T, 8>(a, s)
           : a.H % 4 == 0 ? run_spread<T, 4>(a, s)
           : a.H % 2 == 0 ? run_spread<T, 2>(a, s)
                          : run_spread<T, 1>(a, s);
}

}  // namespace

cudaError_t launch_slots_combine(const SlotsArgs& a, cudaStream_t s) {
    if (a.dtype == STRATA_BF16)
        return a.out_dtype == STRATA_F32 ? pick_combine<__nv_bfloat16, float>(a, s)
                                         : pick_combine<__nv_bfloat16, __nv_bfloat16>(a, s);
    return a.out_dtype == STRATA_F32 ? pick_combine<__half, float>(a, s) : pick_combine<__half, __half>(a, s);
}

cudaError_t launch_slots_spread(const SlotsArgs& a, cudaStream_t s) {
    return a.dtype == STRATA_BF16 ? pick_spread<__nv_bfloat16>(a, s) : pick_spread<__half>(a, s);
}

}  // namespace strata
