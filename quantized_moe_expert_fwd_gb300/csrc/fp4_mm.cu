// fp4_mm.cu -- the grouped product of two 4-bit operands on the tensor cores.
//
// A tile is 128 slots of a group by 128 rows of W, accumulated in tensor
// memory by the block-scaled tcgen05.mma (e2m1 operands, K = 64 an
// instruction, the scales applied by the tensor core), K = 256 a stage: 128
// packed bytes a row with the 128-byte swizzle.  The scales of both operands
// lie in memory as 128-row by 4-scale tiles in the order that the tensor
// memory wants, so a stage's scales are one contiguous bulk copy per operand
// and one tcgen05.cp per tile (32 lanes by 4 words, to all four lane
// quarters).  An NV scale word covers one K step (scale_vec::4X), an MX word
// two (scale_vec::2X, the step's half of the word picked by the descriptor).
//
// Measured, NV, 16384 rows of 256 experts of 1024 x 2048 with SwiGLU: 56 us
// (bytes at the copy's rate 50.5); 131072 rows of 8 experts of 2048 x 2048:
// 286 us, 3.8 PFLOP/s, bound by the 36 KB a stage that every CTA takes from L2.
//
// The accumulator is drained into fp32 registers of the epilogue every 2048
// terms for fp32 outputs, every 8192 for 16-bit ones, for the reason that
// grouped_tc.cu gives: 2^20 terms of one sign in one accumulator came out
// 2.4e-4 (MX) and 3.6e-4 (NV) low.
//
// Roles, buffers and waits as in grouped_tc.cu.  The epilogue multiplies by
// alpha[e] and, for SwiGLU, joins the gate and up columns 2i and 2i + 1, which
// one lane holds side by side.
#include "fp4.cuh"
#include "grouped_tc.cuh"

namespace strata {

namespace {

constexpr int kF4Threads = kGtThreads + 64;     // two warps more: the scales' copies
constexpr int kF4SfWarp = 10;                   // warp 10: A's, 11: B's
constexpr int kF4N = 128;                       // tile columns
constexpr int kF4K = 256;                       // K of a stage
// Stages between drains, for fp32 and for 16-bit outputs.
constexpr int kF4Drain32 = 8, kF4Drain16 = 32;
constexpr uint32_t kF4Data = 128 * 128;         // one operand's packed rows of a stage

template <int FMT>
struct F4 {
    static constexpr int kWords = FMT == 0 ? 2 : 4;            // scale words a stage
    static constexpr uint32_t kSf = kWords * 512;              // one operand's scales of a stage
    static constexpr uint32_t kStage = 2 * kF4Data + 2 * kSf;
    static constexpr int kStages = 5;
    static constexpr size_t kDyn = size_t(kStages) * kStage + kGtStoreBytes + 1024;
    // tensor memory: two accumulators, both operands' scales of every stage
    static constexpr uint32_t kSfCol = 2 * kF4N;
    static constexpr uint32_t kSfCols = kWords * 4;            // one operand's, a stage
    static_assert(kSfCol + kStages * 2 * kSfCols <= 512, "TMEM columns");
};

struct F4Maps {
    GtRowMaps a;
    CUtensorMap b;
};

// Instruction descriptor of the block-scaled kinds with e2m1 operands:
//   [4,6) B scale id  [7,10) A format (1 = e2m1)  [10,12) B format
//   [17,23) N >> 3  [23] scale type (0 = ue4m3, 1 = ue8m0)  [27,29) M >> 7
//   [29,31) A scale id
__device__ __forceinline__ uint32_t idesc_f4(int M, int N, int ue8m0, int sf_id) {
    return (uint32_t(sf_id) << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) |
           (uint32_t(ue8m0) << 23) | (uint32_t(M >> 7) << 27) | (uint32_t(sf_id) << 29);
}

template <int FMT>
__device__ __forceinline__ void umma_f4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if (FMT == 0)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %6, 0; "
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
            "[%5], p; }" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %6, 0; "
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
            "[%4], [%5], p; }" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// One scale tile (512 bytes of shared memory, no swizzle, 8-row groups of
// 128 bytes) to 4 columns of tensor memory, all four lane quarters.
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint32_t smem) {
    const uint64_t d = uint64_t((smem & 0x3FFFFu) >> 4) | (uint64_t(128 >> 4) << 16) |
                       (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// silu(g) u with an exponential that never passes 1: e^-g leaves fp32 (and the
// fast quotient's range before) where g is below -87, the result does not when
// u is large.  Below -87.3 the exponential loses bits, at -104 it is 0.  16-bit
// outputs take the fast exponential and quotient (relative error 2 + 1.2 |g|
// steps of 2^-23, next to roundings of 2^-8 or 2^-11).  Against g / (1 + e^-g):
// 71.8 and 73.4 us for 32768 rows of 8 experts of 2048 x 2048, 55.5 either way
// for a prompt.
template <bool F32>
__device__ __forceinline__ float f4_swiglu(float g, float u) {
    const float e = F32 ? expf(-fabsf(g)) : __expf(-fabsf(g));
    const float n = g < 0.0f ? g * e : g;
    return (F32 ? n / (1.0f + e) : __fdividef(n, 1.0f + e)) * u;
}

// PIECES: the reduction is longer than a piece, a kernel of its own (in one
// with the other, that lost up to 5 %).  Without drains and with them, NV, fp32
// outputs: 32768 rows of 8 experts, 4096 to 1024 columns, 76.8 and 78.5 us.
template <int FMT, bool F32, bool SWIGLU, bool PIECES>
__global__ void __launch_bounds__(kF4Threads, 1)
    k_gmm_f4(const __grid_constant__ F4Maps maps, Fp4GmmArgs a, int vec) {
    using C = F4<FMT>;
    constexpr int PIECE = F32 ? kF4Drain32 : kF4Drain16;
    extern __shared__ uint8_t f4_dyn[];
    __shared__ GroupTable t;
    // full: a stage's copies landed; sf_full: its scales are in tensor memory
    // too; empty: its products are done (shared memory and scales free again)
    __shared__ __align__(8) uint64_t full[C::kStages], sf_full[C::kStages], empty[C::kStages];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], done;
    __shared__ uint32_t tmem_base;
    __shared__ GtStop stop;
    const GtWaits<false> waits{a.err, &stop};
    const int tid = threadIdx.x, lane = tid & 31;
    const int wid = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform to the compiler
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(f4_dyn) + 1023) &
                                               ~uintptr_t(1023));
    // a stage: A rows, B rows (1024-byte aligned); the scales of all stages behind
    uint8_t* sf_base = base + size_t(C::kStages) * 2 * kF4Data;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&sf_full[i], 2);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kGtEpiWarps);
        }
        mbar_init(&done, 1);
        stop = GtStop{};
        mbar_fence_init();
        tma_prefetch_map(&maps.b);
        tma_prefetch_map(&maps.a.part);
    }
    if (wid == kGtMmaWarp) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch();
    pdl_wait();
    build_groups(t, a.offsets, a.E, a.M, kGtRows, a.err);
    const uint32_t tmem = tmem_base;
    const int nt = (a.N + kF4N - 1) / kF4N, words = fp4_words(a.K, FMT);
    const int stages = (a.K + kF4K - 1) / kF4K;
    const int blocks = t.pre[a.E];
    const GtIter<false> first_tile(nt, 0, int(blockIdx.x), int(gridDim.x));

    if (wid == kGtTmaWarp) {
        if (elect_one()) {
            uint32_t st = 0;
            bool ok = true;
            for (auto it = first_tile; ok && it.m < blocks; it.next()) {
                const int rb = it.m, ct = it.c;
                const int e = group_of_block(t, a.E, rb);
                const int in = (rb - t.pre[e]) * kGtRows, arow = t.row[e] + in;
                const int nbox = (min(kGtRows, t.cnt[e] - in) + kGtBox - 1) / kGtBox;
                const bool whole = nbox == kGtRows / kGtBox;
                const CUtensorMap* ma = whole ? &maps.a.whole : &maps.a.part;
                const uint8_t* sa_g = a.xs + size_t(rb) * words * 512;
                const uint8_t* sb_g = a.wsc + (size_t(e) * nt + ct) * words * 512;
                for (int ks = 0; ks < stages; ++ks, ++st) {
                    const uint32_t s = st % C::kStages, round = st / C::kStages;
                    if (round > 0 && !gt_wait(&empty[s], (round - 1) & 1, waits, 60, s)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = base + s * (2 * kF4Data);
                    uint8_t* sf = sf_base + s * (2 * C::kSf);
                    const int w0 = ks * C::kWords;
                    const uint32_t sf_bytes = uint32_t(min(C::kWords, words - w0)) * 512u;
                    mbar_expect_tx(&full[s],
                                   uint32_t(nbox) * kGtBox * 128u + kF4Data + 2 * sf_bytes);
                    tma_load_2d(sa, ma, ks * (kF4K / 2), arow, &full[s]);
                    if (!whole)
                        for (int j = 1; j < nbox; ++j)
                            tma_load_2d(sa + j * (kGtBox * 128), ma, ks * (kF4K / 2),
                                        arow + j * kGtBox, &full[s]);
                    tma_load_3d(sa + kF4Data, &maps.b, ks * (kF4K / 2), ct * kF4N, e, &full[s]);
                    bulk_g2s(sf, sa_g + size_t(w0) * 512, sf_bytes, &full[s]);
                    bulk_g2s(sf + C::kSf, sb_g + size_t(w0) * 512, sf_bytes, &full[s]);
                }
            }
            // every copy has landed and has been consumed before the CTA exits
            const uint32_t tail = st > C::kStages ? st - C::kStages : 0;
            for (uint32_t k = tail; ok && k < st; ++k)
                ok = gt_wait(&empty[k % C::kStages], (k / C::kStages) & 1, waits, 61, k % C::kStages);
            if (!ok) {
                // a wait ran out: the copies have landed
                waits.mark(&stop.halted, 1u);
                for (uint32_t k = tail; k < st; ++k)
                    mbar_wait(&full[k % C::kStages], (k / C::kStages) & 1);
            }
        }
    } else if (wid >= kF4SfWarp) {
        // one operand's scales of each stage to tensor memory, on a thread of
        // their own: a copy takes about as long to issue as a product
        if (elect_one()) {
            const int op = wid - kF4SfWarp;
            uint32_t st = 0;
            for (auto it = first_tile; it.m < blocks; it.next()) {
                for (int ks = 0; ks < stages; ++ks, ++st) {
                    const uint32_t s = st % C::kStages;
                    gt_wait<false, true>(&full[s], (st / C::kStages) & 1, waits, 66 + op, s);
                    tc_fence_after();
                    const uint32_t sf = smem_u32(sf_base + s * (2 * C::kSf) + op * C::kSf);
                    const uint32_t col = tmem + C::kSfCol + (2 * s + op) * C::kSfCols;
                    const int nw = min(C::kWords, words - ks * C::kWords);
#pragma unroll
                    for (int w = 0; w < C::kWords; ++w)
                        if (w < nw) sf_copy(col + 4 * w, sf + w * 512);
                    umma_commit(&sf_full[s]);
                }
            }
        }
    } else if (wid == kGtMmaWarp) {
        uint32_t st = 0, acc = 0;
        for (auto it = first_tile; it.m < blocks; it.next(), ++acc) {
            auto free_acc = [&]() {
                if (acc >= 2)
                    gt_wait<false, true>(&acc_empty[acc & 1u], ((acc >> 1) - 1) & 1, waits, 62,
                                         acc & 1u);
            };
            free_acc();
            for (int ks = 0; ks < stages; ++ks, ++st) {
                const int nth = PIECES ? ks % PIECE : ks;      // of the piece
                const bool last = ks == stages - 1 || (PIECES && nth == PIECE - 1);
                if (PIECES && ks > 0 && nth == 0) {
                    ++acc;
                    free_acc();
                }
                const uint32_t buf = acc & 1u;
                const uint32_t s = st % C::kStages;
                gt_wait<false, true>(&sf_full[s], (st / C::kStages) & 1, waits, 63, s);
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sa = smem_u32(base + s * (2 * kF4Data));
                    const uint32_t ca = tmem + C::kSfCol + s * (2 * C::kSfCols);
                    const uint32_t cb = ca + C::kSfCols;
                    // K steps that exist: past K the scales are not loaded
                    const int steps = min(4, (a.K - ks * kF4K + 63) / 64);
                    const uint64_t da = sdesc_k_sw128(sa), db = sdesc_k_sw128(sa + kF4Data);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < steps) {
                            const int w = FMT == 0 ? j / 2 : j;
                            umma_f4<FMT>(tmem + buf * kF4N, da + 2 * j, db + 2 * j,
                                         idesc_f4(kGtRows, kF4N, FMT == 0, FMT == 0 ? 2 * (j & 1) : 0),
                                         ca + 4 * w, cb + 4 * w, (nth | j) != 0 ? 1u : 0u);
                        }
                    umma_commit(&empty[s]);
                    if (last) umma_commit(&acc_full[buf]);
                }
                __syncwarp();
            }
        }
        // no product may still be writing the TMEM when it is freed
        if (elect_one()) umma_commit(&done);
        __syncwarp();
        gt_wait<false, false, false>(&done, 0, waits, 64, 0);
    } else if (wid < kGtEpiWarps) {
        const int half = wid >> 2, r = (wid & 3) * 32 + lane;
        const uint32_t tl = tmem + (uint32_t((wid & 3) * 32) << 16) + uint32_t(half * (kF4N / 2));
        const int cols = SWIGLU ? a.N / 2 : a.N;
        uint32_t* stage =
            reinterpret_cast<uint32_t*>(sf_base + C::kStages * 2 * C::kSf) + wid * kGtStoreWords;
        uint32_t acc = 0;
        for (auto it = first_tile; it.m < blocks; it.next()) {
            const int rb = it.m, ct = it.c;
            const int e = group_of_block(t, a.E, rb);
            const int in = (rb - t.pre[e]) * kGtRows;
            const bool live = r < t.cnt[e] - in;
            const float al = a.alpha != nullptr ? __ldg(a.alpha + e) : 1.0f;
            // the warp's rows, and the first one's place
            const int rows = t.cnt[e] - in - (r - lane);
            const size_t row = size_t(t.row[e] + in + r - lane) * cols;
            // piece c of 32 columns, from its sums
            auto finish = [&](int c, const float* p) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = live ? al * p[j] : 0.0f;
                const int c0 = ct * kF4N + half * (kF4N / 2) + c * 32;
                if (SWIGLU) {
                    float h[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) h[j] = f4_swiglu<F32>(v[2 * j], v[2 * j + 1]);
                    gt_store<F32, 16>(a.out, row + c0 / 2, cols, min(rows, 32), h, cols - c0 / 2, vec,
                                      a.out_dtype == STRATA_BF16, stage);
                } else {
                    gt_store<F32, 32>(a.out, row + c0, cols, min(rows, 32), v, cols - c0, vec,
                                      a.out_dtype == STRATA_BF16, stage);
                }
            };
            auto taken = [&](uint32_t buf) {             // the accumulator is free again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[buf]);
            };
            // warps whose rows all lie behind the group's end have nothing to do
            // but to free the accumulators
            if constexpr (!PIECES) {                     // stored as it is read
                const uint32_t buf = acc & 1u;
                gt_wait(&acc_full[buf], (acc >> 1) & 1, waits, 65, buf);
                tc_fence_after();
                if (rows > 0)
#pragma unroll
                    for (int c = 0; c < kF4N / 64; ++c) {
                        uint32_t u[32];
                        tmem_ld32(tl + buf * kF4N + c * 32, u);
                        tmem_ld_wait();
                        finish(c, reinterpret_cast<const float*>(u));
                    }
                taken(buf);
                ++acc;
            } else {
                float sum[kF4N / 64][32];
#pragma unroll
                for (int c = 0; c < kF4N / 64; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
                for (int ks = 0; ks < stages; ks += PIECE, ++acc) {
                    const uint32_t buf = acc & 1u;
                    gt_wait(&acc_full[buf], (acc >> 1) & 1, waits, 65, buf);
                    tc_fence_after();
                    if (rows > 0)
#pragma unroll
                        for (int c = 0; c < kF4N / 64; ++c) {
                            uint32_t u[32];
                            tmem_ld32(tl + buf * kF4N + c * 32, u);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j) sum[c][j] += __uint_as_float(u[j]);
                        }
                    taken(buf);
                }
                if (rows > 0)
#pragma unroll
                    for (int c = 0; c < kF4N / 64; ++c) finish(c, sum[c]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // a wait ran out: scales may still be on their way to tensor memory
    if (!waits.seen(&stop.stop, 0u)) gt_settle();
    tc_fence_after();
    if (wid == kGtMmaWarp) tmem_dealloc(tmem, 512);
}

template <int FMT, bool F32, bool SWIGLU>
cudaError_t f4_run(const Fp4GmmArgs& g, cudaStream_t s) {
    F4Maps m;
    const bool ok = gt_map(&m.b, 1, g.wq, g.K / 2, g.N, g.E, kF4N) &&
                    gt_map(&m.a.part, 1, g.xq, g.K / 2, g.M, 0, kGtBox) &&
                    gt_map(&m.a.whole, 1, g.xq, g.K / 2, g.M, 0, kGtRows);
    if (!ok) return cudaErrorInvalidValue;
    const int vec = gt_vec(g.out, size_t(SWIGLU ? g.N / 2 : g.N) * (F32 ? 4 : 2));
    const int sms = device_info().sms;
    if (g.K > (F32 ? kF4Drain32 : kF4Drain16) * kF4K)
        return gt_launch<k_gmm_f4<FMT, F32, SWIGLU, true>>(kF4Threads, 1, sms, F4<FMT>::kDyn, s, m, g,
                                                           vec);
    return gt_launch<k_gmm_f4<FMT, F32, SWIGLU, false>>(kF4Threads, 1, sms, F4<FMT>::kDyn, s, m, g,
                                                        vec);
}

template <int FMT>
cudaError_t f4_pick(const Fp4GmmArgs& g, cudaStream_t s) {
    if (g.out_dtype == STRATA_F32)
        return g.swiglu ? f4_run<FMT, true, true>(g, s) : f4_run<FMT, true, false>(g, s);
    return g.swiglu ? f4_run<FMT, false, true>(g, s) : f4_run<FMT, false, false>(g, s);
}

}  // namespace

cudaError_t launch_grouped_mm_fp4(const Fp4GmmArgs& g, cudaStream_t s) {
    return g.fmt == STRATA_FP4_MX ? f4_pick<0>(g, s) : f4_pick<1>(g, s);
}

}  // namespace strata
