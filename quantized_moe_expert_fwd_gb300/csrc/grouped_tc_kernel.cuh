// grouped_tc_kernel.cuh -- the grouped products on the tensor cores.
//
// A tile is 128 rows by BN columns of the output, accumulated in tensor
// memory by tcgen05.mma (fp32) over the whole reduction, 64 of it a pipeline
// stage:
//   forward  rows: slots of a group     columns: n   reduction: k
//   dx       rows: slots of a group     columns: k   reduction: n
//   dw       rows: n of an expert       columns: k   reduction: the group's slots
// Operands come by TMA with the 128-byte swizzle.  An operand whose rows run
// along the reduction (W in dx, dy and x in dw) lands as sub-blocks of 64
// columns by 64 reduction rows and is read MN-major.  Row tiles start at a
// group's first row, so a box may reach into the next group: in forward and
// dx those rows only feed accumulator rows that are not stored; in dw they
// are reduction rows, and the last stage's are overwritten with zeros in both
// operands before the MMA (a product with zero alone would let an infinity
// of the next group through).
//
// Persistent, one CTA of 10 warps per SM: warps 0..7 epilogue (warp w: lanes
// 32 (w % 4) .. of column half w / 4), 8 TMA producer, 9 MMA.  Two
// accumulator buffers, so a tile's epilogue overlaps the next tile's MMAs.
// Long groups' tiles are made by pairs of CTAs, and few tiles' reductions are
// split over a cluster (gt_pick has the rules and what they measured).
//
// Measured, 256 experts of 1024 x 2048 in bf16, 16384 rows (us; bytes at the
// copy's rate 175.6): forward 184, dx 173, dw 199; 65536 rows into 32 experts,
// dw in fp32: 200 in a captured graph, 220 as calls with changing inputs (FLOPs
// at the burst rate 144.7).
//
// The tensor cores truncate as they add, so terms of one sign lose about 1e-7
// of the sum with every 16 of them (16-bit outputs of 2^18 such terms in one
// accumulator: 1.7e-3 off).  The accumulator is therefore drained into fp32
// registers of the epilogue, where the pieces are added with rounding: every
// 512 terms for fp32 outputs, every 2048 for 16-bit ones (a loss of 1.3e-5,
// next to half steps of 4.9e-4 and 3.9e-3).
#pragma once

#include <type_traits>

#include "grouped_tc.cuh"

namespace strata {

namespace {

constexpr int kGtK = 64;                        // reduction of a stage (128 bytes)
// What a kernel writes: 16-bit outputs of a reduction of one piece, of any
// number of pieces, and fp32.  (Forward with the single-piece kernel and with
// the other, 32 experts of 1024 x 2048: 28.4 and 29.1 us at 64 rows a group,
// 31.9 and 32.7 at 128, 58.4 and 59.2 at 512.)
constexpr int kGt16 = 0, kGt16Pieces = 1, kGt32 = 2;
// Stages of a piece (between two drains), for fp32 and for 16-bit outputs.
constexpr int kGtDrain32 = 8, kGtDrain16 = 32;
constexpr uint32_t kGtABytes = kGtRows * 128;
constexpr uint32_t kGtSub = 64 * 128;           // a 64 x 64 MN-major sub-block

// dw writes a whole tile for every stage or two that it reads: it gives up a
// stage for the output's staging, a piece of 32 rows by 128 bytes an epilogue
// warp.  (Two pieces: no faster where they fit, 196 us instead of 193 for
// 16384 rows into 256 experts; in a pair they cost another stage, 215 instead
// of 202 for 65536 rows.)
constexpr uint32_t kGtPiece = 32 * 128;

constexpr int kGtPair = 1, kGtSplit = 2;        // what the CTAs of a cluster share

// A kernel's geometry.  CL = kGtPair: two CTAs make one tile of 256 rows by
// BN columns; each loads its 128 rows and half of the columns.  CL =
// kGtSplit: the CTAs of a cluster take a part of one tile's reduction each.
template <int MODE, int BN, int CL, uint32_t STAGING = kGtStoreBytes>
struct Gt {
    static constexpr bool PAIR = CL == kGtPair;
    static constexpr int kCols = PAIR ? BN / 2 : BN;             // B columns a CTA loads
    static constexpr uint32_t kBBytes = uint32_t(kCols) * 128u;
    static constexpr uint32_t kStage = kGtABytes + kBBytes;
    static constexpr uint32_t kStagingBytes = MODE == kGmmDw ? kGtEpiWarps * kGtPiece : STAGING;
    static constexpr int kStages = int((214016u - kStagingBytes) / kStage);
    static constexpr size_t kDyn = size_t(kStages) * kStage + kStagingBytes + 1024;
    static constexpr int kBlock = PAIR ? 2 * kGtRows : kGtRows;  // rows of a tile
};

struct GtMaps {
    GtRowMaps a;                                // dw: 64-row boxes in both
    CUtensorMap b;
    CUtensorMap out;                            // dw alone
};

struct GtArgs {
    void* out;
    const int32_t* offsets;
    uint32_t* err;
    int M, K, N, E;
    int bf16;                                   // operands (and a 16-bit output)
    int vec;                                    // bytes that every output row is aligned to: 32, 16, 0
};

// k0, k1: the stages of the reduction that this CTA takes.
struct GtTile {
    int e, arow, rows, c0, k0, k1, slot0, cnt;
    size_t orow;
};
constexpr int kGtPartPitch = 132;               // split: floats of a row of partial sums

// rank: the CTA's half of a pair's rows, or its part of the reduction.
template <int MODE, int BN, int CL>
__device__ __forceinline__ GtTile gt_tile(const GroupTable& t, const GtArgs& a,
                                          const GtIter<MODE == kGmmDw>& it, int rank) {
    constexpr int BLOCK = Gt<MODE, BN, CL>::kBlock;
    const int half = CL == kGtPair ? rank * kGtRows : 0;
    GtTile i;
    i.c0 = it.c * BN;
    int stages;
    if (MODE == kGmmDw) {
        i.e = it.e;
        i.arow = it.m * BLOCK + half;
        i.rows = min(kGtRows, a.N - i.arow);
        i.slot0 = t.row[i.e];
        i.cnt = t.cnt[i.e];
        stages = (i.cnt + kGtK - 1) / kGtK;
        i.orow = size_t(i.e) * a.N + i.arow;
    } else {
        i.e = group_of_block(t, a.E, it.m);
        const int in = (it.m - t.pre[i.e]) * BLOCK + half;
        i.arow = t.row[i.e] + in;
        i.rows = min(kGtRows, t.cnt[i.e] - in);
        i.slot0 = i.cnt = 0;
        stages = ((MODE == kGmmFwd ? a.K : a.N) + kGtK - 1) / kGtK;
        i.orow = size_t(i.arow);
    }
    i.k0 = 0;
    i.k1 = stages;
    if (CL == kGtSplit) {
        const int part = (stages + int(cluster_size()) - 1) / int(cluster_size());
        i.k0 = min(rank * part, stages);
        i.k1 = min(i.k0 + part, stages);
    }
    return i;
}

// dw: the rows of stage ks that the last 16-row step takes from behind the
// group's end.
template <int MODE>
__device__ __forceinline__ int gt_dead(const GtTile& i, int ks) {
    return MODE == kGmmDw ? -min(kGtK, i.cnt - ks * kGtK) & 15 : 0;
}

// Split: 32 partial sums to shared memory.
__device__ __forceinline__ void gt_part(float* p, const float* v) {
#pragma unroll
    for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
}

// What becomes of the sums: the output as it is (GtPlain), or an epilogue EPI
// (16-bit outputs of forward and dx).  It takes 32 columns of a warp's 32
// rows at a time,
//   take(read ahead, first row, rows, first column, end, values, the warp's
//        staging),
// or, where a reduction was split, four columns of a row a lane,
//   quad(row, first column, values, whether they exist),
// and reads ahead of a tile's sums,
//   ahead(first row, rows, first column, end, the warp's staging),
// which has kWarpStaging bytes.
// Its steps are a loop that is not unrolled, over sums in tensor memory (where
// pieces were added they go back there first): unrolled, the code of SwiGLU's
// gradient left the instruction cache (2048-token prompt 201 us).
struct GtPlain {
    static constexpr uint32_t kWarpStaging = kGtStoreWords * 4;
};

template <int MODE, int BN, int OUT, int CL, typename EPI = GtPlain>
__global__ void __launch_bounds__(kGtThreads, 1)
    k_gmm_tc(const __grid_constant__ GtMaps maps, GtArgs a, EPI epi) {
    constexpr bool PLAIN = std::is_same<EPI, GtPlain>::value;
    using G = Gt<MODE, BN, CL, kGtEpiWarps * EPI::kWarpStaging>;
    constexpr bool PAIR = CL == kGtPair, SPLIT = CL == kGtSplit;
    constexpr int STAGES = G::kStages;
    constexpr bool F32 = OUT == kGt32, PIECES = OUT != kGt16;
    constexpr int PIECE = F32 ? kGtDrain32 : kGtDrain16;
    constexpr uint32_t STAGE = G::kStage;
    extern __shared__ uint8_t gt_dyn[];
    __shared__ GroupTable t;
    // full: a stage's copies landed.  Pairs: both CTAs' copies complete on rank
    // 0's `both`; a stage that needs rows overwritten instead completes on each
    // CTA's own `full`, and rank 1 reports at rank 0's `fixed` (a report from
    // thread to thread takes a microsecond, so only those stages pay it).
    // empty, acc_full and done signal in both CTAs, acc_empty at rank 0.
    __shared__ __align__(8) uint64_t full[STAGES], empty[STAGES], both[STAGES], fixed[STAGES];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], done;
    __shared__ uint32_t tmem_base, pieces;
    __shared__ GtStop stop;
    const GtWaits<PAIR> waits{a.err, &stop};
    const int tid = threadIdx.x, lane = tid & 31;
    const int wid = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform to the compiler
    const int rank = CL != 0 ? int(cluster_rank()) : 0;
    const int workers = CL != 0 ? int(cluster_size()) : 1;       // CTAs of a tile
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gt_dyn) + 1023) &
                                               ~uintptr_t(1023));
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&both[i], 1);
            mbar_init(&fixed[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], PAIR ? 2 * kGtEpiWarps : kGtEpiWarps);
        }
        mbar_init(&done, 1);
        stop = GtStop{};
        mbar_fence_init();
        tma_prefetch_map(&maps.b);
        tma_prefetch_map(&maps.a.part);
    }
    if (wid == kGtMmaWarp) {
        if (PAIR) {
            tmem_alloc2(&tmem_base, 2 * BN);
            tmem_relinquish2();
        } else {
            tmem_alloc(&tmem_base, 2 * BN);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();            // both CTAs' barriers exist
    tc_fence_after();
    pdl_launch();
    pdl_wait();
    build_groups(t, a.offsets, a.E, a.M, G::kBlock, a.err);
    const uint32_t tmem = tmem_base;
    const int cols = MODE == kGmmFwd ? a.N : a.K;
    const GtIter<MODE == kGmmDw> first_tile(
        (cols + BN - 1) / BN, (a.N + G::kBlock - 1) / G::kBlock,
        int(blockIdx.x) / workers, int(gridDim.x) / workers);
    const int blocks = t.pre[a.E];
    auto more = [&](const GtIter<MODE == kGmmDw>& it) {
        return MODE == kGmmDw ? it.e < a.E : it.m < blocks;
    };

    if (wid == kGtTmaWarp) {
        if (elect_one()) {
            uint32_t st = 0;
            bool ok = true;
            for (auto it = first_tile; ok && more(it); it.next()) {
                const GtTile i = gt_tile<MODE, BN, CL>(t, a, it, rank);
                // a pair always loads whole boxes, so that rank 0 knows the bytes of both
                const int nbox = PAIR || MODE == kGmmDw ? kGtRows / kGtBox
                                                        : (i.rows + kGtBox - 1) / kGtBox;
                const bool whole = nbox == kGtRows / kGtBox;
                const CUtensorMap* ma = whole ? &maps.a.whole : &maps.a.part;
                const int b0 = i.c0 + (PAIR ? rank * G::kCols : 0);
                const uint32_t bytes = uint32_t(nbox) * kGtBox * 128u + G::kBBytes;
                for (int ks = i.k0; ks < i.k1; ++ks, ++st) {
                    const uint32_t s = st % STAGES, round = st / STAGES;
                    if (round > 0 && !gt_wait(&empty[s], (round - 1) & 1, waits, 50, s)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = base + s * STAGE;
                    uint8_t* sb = sa + kGtABytes;
                    const int r0 = ks * kGtK;
                    if (PAIR && !gt_dead<MODE>(i, ks)) {
                        const uint32_t bar = rank0_addr(&both[s]);
                        if (rank == 0) mbar_expect_tx(&both[s], 2 * bytes);
                        if (MODE == kGmmDw) {
                            for (int j = 0; j < 2; ++j)
                                tma2_load_2d(sa + j * kGtSub, ma, i.arow + 64 * j, i.slot0 + r0, bar);
                            for (int j = 0; j < G::kCols / 64; ++j)
                                tma2_load_2d(sb + j * kGtSub, &maps.b, b0 + 64 * j, i.slot0 + r0, bar);
                        } else {
                            tma2_load_2d(sa, ma, r0, i.arow, bar);
                            if (MODE == kGmmFwd) {
                                tma2_load_3d(sb, &maps.b, r0, b0, i.e, bar);
                            } else {
                                for (int j = 0; j < G::kCols / 64; ++j)
                                    tma2_load_3d(sb + j * kGtSub, &maps.b, b0 + 64 * j, r0, i.e, bar);
                            }
                        }
                        continue;
                    }
                    mbar_expect_tx(&full[s], bytes);
                    if (MODE == kGmmDw) {
                        for (int j = 0; j < 2; ++j)
                            tma_load_2d(sa + j * kGtSub, ma, i.arow + 64 * j, i.slot0 + r0, &full[s]);
                        for (int j = 0; j < G::kCols / 64; ++j)
                            tma_load_2d(sb + j * kGtSub, &maps.b, b0 + 64 * j, i.slot0 + r0,
                                        &full[s]);
                    } else {
                        tma_load_2d(sa, ma, r0, i.arow, &full[s]);
                        if (!whole)
                            for (int j = 1; j < nbox; ++j)
                                tma_load_2d(sa + j * (kGtBox * 128), ma, r0, i.arow + j * kGtBox,
                                            &full[s]);
                        if (MODE == kGmmFwd) {
                            tma_load_3d(sb, &maps.b, r0, b0, i.e, &full[s]);
                        } else {
                            for (int j = 0; j < G::kCols / 64; ++j)
                                tma_load_3d(sb + j * kGtSub, &maps.b, b0 + 64 * j, r0, i.e,
                                            &full[s]);
                        }
                    }
                }
            }
            // every copy has landed, has been consumed, and the MMAs' arrivals are
            // here, before the CTA exits
            const uint32_t tail = st > STAGES ? st - STAGES : 0;
            for (uint32_t k = tail; ok && k < st; ++k)
                ok = gt_wait(&empty[k % STAGES], (k / STAGES) & 1, waits, 51, k % STAGES);
            if (!ok) {
                // a wait ran out: the copies have landed (a pair's second CTA's
                // report to the first)
                waits.mark(&stop.halted, 1u << rank);
                for (uint32_t k = tail; !PAIR && k < st; ++k)
                    mbar_wait(&full[k % STAGES], (k / STAGES) & 1);
                gt_settle();
            }
        }
    } else if (wid == kGtMmaWarp) {
        const uint32_t idesc = idesc_f16(G::kBlock, BN, a.bf16) |
                               (MODE == kGmmDw ? kIdescMnA : 0u) |
                               (MODE != kGmmFwd ? kIdescMnB : 0u);
        constexpr uint32_t a_step = MODE == kGmmDw ? 2048 / 16 : 2;
        constexpr uint32_t b_step = MODE != kGmmFwd ? 2048 / 16 : 2;
        uint32_t st = 0, acc = 0;
        uint32_t both_phase = 0, own_phase = 0;      // a bit a stage: the phase waited for next
        for (auto it = first_tile; more(it); it.next()) {
            const GtTile i = gt_tile<MODE, BN, CL>(t, a, it, rank);
            for (int ks = i.k0; ks < i.k1; ++ks, ++st) {
                const uint32_t s = st % STAGES;
                const int nth = ks - i.k0;
                const bool first = PIECES ? nth % PIECE == 0 : nth == 0;
                const bool last = ks == i.k1 - 1 || (PIECES && nth % PIECE == PIECE - 1);
                const uint32_t buf = acc & 1u;
                if ((!PAIR || rank == 0) && first && acc >= 2)
                    gt_wait<PAIR, true>(&acc_empty[buf], ((acc >> 1) - 1) & 1, waits, 52, buf);
                uint8_t* sa = base + s * STAGE;
                uint8_t* sb = sa + kGtABytes;
                const int dead = gt_dead<MODE>(i, ks);         // rows of the next group
                int steps = kGtK / 16;
                if (MODE == kGmmDw) steps = (min(kGtK, i.cnt - ks * kGtK) + 15) / 16;
                if (!PAIR) {
                    gt_wait<false, true>(&full[s], (st / STAGES) & 1, waits, 53, s);
                } else if (dead == 0) {
                    if (rank == 0) {
                        gt_wait<false, true>(&both[s], (both_phase >> s) & 1u, waits, 56, s);
                        both_phase ^= 1u << s;
                    }
                } else {
                    gt_wait<false, true>(&full[s], (own_phase >> s) & 1u, waits, 53, s);
                }
                if (dead > 0) {
                    const int valid = steps * 16 - dead;
                    for (int j = lane; j < dead * 8 * (2 + G::kCols / 64); j += 32) {
                        const int sub = j / (dead * 8), r = j % (dead * 8);
                        *reinterpret_cast<uint4*>(sa + sub * kGtSub + valid * 128 + r * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    if (PAIR) {
                        fence_proxy_async_all();
                        __syncwarp();
                        if (rank == 0)
                            gt_wait<true, true>(&fixed[s], (own_phase >> s) & 1u, waits, 57, s);
                        else if (elect_one()) mbar_arrive_rank0(&fixed[s]);
                        own_phase ^= 1u << s;
                    } else {
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                }
                if (PAIR && rank != 0) {
                    if (last) ++acc;
                    continue;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t da = MODE == kGmmDw ? sdesc_mn_sw128(smem_u32(sa), kGtSub)
                                                       : sdesc_k_sw128(smem_u32(sa));
                    const uint64_t db = MODE != kGmmFwd ? sdesc_mn_sw128(smem_u32(sb), kGtSub)
                                                        : sdesc_k_sw128(smem_u32(sb));
#pragma unroll
                    for (int j = 0; j < kGtK / 16; ++j)
                        if (MODE != kGmmDw || j < steps) {
                            const uint32_t add = (first && j == 0) ? 0u : 1u;
                            if (PAIR)
                                umma2_f16(tmem + buf * BN, da + j * a_step, db + j * b_step, idesc, add);
                            else
                                umma_f16(tmem + buf * BN, da + j * a_step, db + j * b_step, idesc, add);
                        }
                    if (PAIR) {
                        umma2_commit(&empty[s]);
                        if (last) umma2_commit(&acc_full[buf]);
                    } else {
                        umma_commit(&empty[s]);
                        if (last) umma_commit(&acc_full[buf]);
                    }
                }
                __syncwarp();
                if (last) ++acc;
            }
        }
        if ((!PAIR || rank == 0) && elect_one()) {
            if (PAIR) umma2_commit(&done);
            else umma_commit(&done);
        }
        __syncwarp();
        // no product may still be writing the TMEM when it is freed
        if (!PAIR) gt_wait<false, false, false>(&done, 0, waits, 54, 0);
        else if (lane == 0) pieces = acc;
    } else {
        constexpr int CH = BN / 64;              // 32-column pieces of a warp's half
        const int half = wid >> 2, r = (wid & 3) * 32 + lane;
        const uint32_t tl = tmem + (uint32_t((wid & 3) * 32) << 16) + uint32_t(half * (BN / 2));
        uint8_t* stage = base + STAGES * STAGE + wid * kGtPiece;            // dw
        uint32_t* store =                                                   // forward, dx
            reinterpret_cast<uint32_t*>(base + STAGES * STAGE + wid * EPI::kWarpStaging);
        // split: this CTA's partial sums, in the stages (all consumed by then)
        float* part = reinterpret_cast<float*>(base) + r * kGtPartPitch + half * (BN / 2);
        uint32_t acc = 0;
        // dw: 128 bytes of each of the warp's 32 rows to memory by TMA, which
        // writes whole lines (32-byte stores of a lane a row: 304 us instead of
        // 193 for 16384 rows into 256 experts); the lanes' 16-byte pieces are spread by the swizzle
        auto put = [&](const GtTile& i, int col, const uint32_t (&w)[32]) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                    make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            const int y = i.arow + (wid & 3) * 32;
            if (lane == 0) {
                if (col < a.K && y < a.N) tma_store_3d(&maps.out, stage, col, y, i.e);
                bulk_commit();
            }
        };
        for (auto it = first_tile; more(it); it.next()) {
            const GtTile i = gt_tile<MODE, BN, CL>(t, a, it, rank);
            const int c0 = i.c0 + half * (BN / 2);
            const size_t at = (i.orow + r - lane) * size_t(cols) + c0;
            const int live = min(32, i.rows - (r - lane));       // of the warp's rows
            auto taken = [&](uint32_t buf) {             // the accumulator is free again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_rank0(&acc_empty[buf]);
                    else mbar_arrive(&acc_empty[buf]);
                }
            };
            if constexpr (!PLAIN && !SPLIT) {
                const int last = min(cols, c0 + BN / 2);
                auto read = epi.ahead(i.orow + r - lane, live, c0, last, store);
                uint32_t buf = acc & 1u;
                gt_wait(&acc_full[buf], (acc >> 1) & 1, waits, 55, buf);
                tc_fence_after();
                if (PIECES && i.k1 - i.k0 > PIECE) {
                    float sum[CH][32];
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
                    for (int ks = i.k0;; ks += PIECE) {
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            uint32_t v[32];
                            tmem_ld32(tl + buf * BN + c * 32, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j) sum[c][j] += __uint_as_float(v[j]);
                        }
                        if (ks + PIECE >= i.k1) break;
                        taken(buf);
                        ++acc;
                        buf = acc & 1u;
                        gt_wait(&acc_full[buf], (acc >> 1) & 1, waits, 55, buf);
                        tc_fence_after();
                    }
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        tmem_st32(tl + buf * BN + c * 32, reinterpret_cast<const uint32_t(&)[32]>(sum[c]));
                    tmem_st_wait();
                }
#pragma unroll 1
                for (int c = 0; c < BN / 2; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(tl + buf * BN + c, v);
                    tmem_ld_wait();
                    epi.take(read, i.orow + r - lane, live, c0 + c, last, reinterpret_cast<const float*>(v),
                             store);
                }
                taken(buf);
                ++acc;
                continue;
            }
            // Stored as it is read: a reduction of one piece, and dw's tiles of one
            // (8 experts of 4096 x 4096, 400 rows each: 109 us, by way of the sums
            // 112).  A pair's go through the sums, so that the accumulator is free
            // before the stores (512 rows a group: 54 us instead of 60).
            constexpr bool DW1 = MODE == kGmmDw && !F32 && !PAIR;
            uint32_t w[32];                      // dw in 16 bits: 64 columns, packed
            auto pack = [&](int c, const float* v) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    w[16 * (c & 1) + j] = gt_pack(v[2 * j], v[2 * j + 1], a.bf16);
                if (c & 1) put(i, c0 + (c - 1) * 32, w);
            };
            if (!PIECES || (DW1 && i.k1 - i.k0 <= PIECE)) {
                const uint32_t buf = acc & 1u;
                if (i.k1 > i.k0) {
                    gt_wait(&acc_full[buf], (acc >> 1) & 1, waits, 55, buf);
                    tc_fence_after();
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint32_t v[32];
                    if (i.k1 > i.k0) {
                        tmem_ld32(tl + buf * BN + c * 32, v);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
                    const float* f = reinterpret_cast<const float*>(v);
                    if (DW1) pack(c, f);
                    else if (SPLIT) gt_part(part + c * 32, f);
                    else if constexpr (PLAIN)
                        gt_store<false, 32>(a.out, at + c * 32, cols, live, f, cols - c0 - c * 32,
                                            a.vec, a.bf16, store);
                }
                if (i.k1 > i.k0) {
                    taken(buf);
                    ++acc;
                }
            } else if constexpr (PIECES) {
                float sum[CH][32];
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
                for (int ks = i.k0; ks < i.k1; ks += PIECE, ++acc) {
                    const uint32_t buf = acc & 1u;
                    gt_wait(&acc_full[buf], (acc >> 1) & 1, waits, 55, buf);
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        uint32_t v[32];
                        tmem_ld32(tl + buf * BN + c * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c][j] += __uint_as_float(v[j]);
                    }
                    taken(buf);
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (MODE == kGmmDw && F32)
                        put(i, c0 + c * 32, reinterpret_cast<const uint32_t(&)[32]>(sum[c]));
                    else if (MODE == kGmmDw) pack(c, sum[c]);
                    else if (SPLIT) gt_part(part + c * 32, sum[c]);
                    else if constexpr (PLAIN)
                        gt_store<F32, 32>(a.out, at + c * 32, cols, live, sum[c], cols - c0 - c * 32,
                                          a.vec, a.bf16, store);
                }
            }
        }
        if (MODE == kGmmDw && lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR && wid == kGtMmaWarp) {
        // A pair waits for its products only here, where the other roles are done:
        // rank 0 issues rank 1's, and a call may last longer than one wait.
        gt_wait<true, false, false>(&done, 0, waits, 54, 0);
        // The other CTA's last arrivals at acc_empty have to be here too before
        // this CTA exits: one under way then would count on a barrier of the
        // CTA that follows it on the SM.
        if (rank == 0)
            for (uint32_t k = pieces > 2 ? pieces - 2 : 0; k < pieces; ++k)
                gt_wait<true, false, false>(&acc_empty[k & 1u], (k >> 1) & 1, waits, 58, k & 1u);
    }
    if (SPLIT) {
        // the partial sums of all parts, added in their order; this CTA
        // stores its share of the tile's rows, a warp 128 columns of one row
        cluster_sync();
        if (more(first_tile)) {
            const GtTile i = gt_tile<MODE, BN, CL>(t, a, first_tile, rank);
            const float* part = reinterpret_cast<const float*>(base);
            const int share = kGtRows / workers, c = i.c0 + lane * 4;
            for (int r = rank * share + wid; r < min(i.rows, (rank + 1) * share);
                 r += kGtThreads / 32) {
                if (PLAIN && c >= cols) continue;
                float v[4] = {};
                for (int p = 0; p < workers; ++p) {
                    const float4 x = ld_cluster_f4(part + r * kGtPartPitch + lane * 4, p);
                    v[0] += x.x;
                    v[1] += x.y;
                    v[2] += x.z;
                    v[3] += x.w;
                }
                if constexpr (!PLAIN) {
                    epi.quad(i.orow + r, c, v, c < cols);
                    continue;
                }
                const size_t at = (i.orow + r) * size_t(cols) + c;
                if (F32) {
                    float* o = static_cast<float*>(a.out) + at;
                    if (a.vec && c + 4 <= cols)
                        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
                    else
                        for (int j = 0; j < min(4, cols - c); ++j) o[j] = v[j];
                } else {
                    uint16_t* o = static_cast<uint16_t*>(a.out) + at;
                    const uint2 w = make_uint2(gt_pack(v[0], v[1], a.bf16), gt_pack(v[2], v[3], a.bf16));
                    if (a.vec && c + 4 <= cols) *reinterpret_cast<uint2*>(o) = w;
                    else
                        for (int j = 0; j < min(4, cols - c); ++j)
                            o[j] = uint16_t((j < 2 ? w.x : w.y) >> (16 * (j & 1)));
                }
            }
        }
    }
    if (CL != 0) cluster_sync();         // the other CTAs read and signal no more
    tc_fence_after();
    if (wid == kGtMmaWarp) {
        if (PAIR) tmem_dealloc2(tmem, 2 * BN);
        else tmem_dealloc(tmem, 2 * BN);
    }
}

// ------------------------------------------------------------------- host
template <int MODE, int BN, int OUT, int CL, typename EPI>
cudaError_t gt_run(const GmmArgs& g, int cluster, int grid, const EPI& epi, cudaStream_t s) {
    using G = Gt<MODE, BN, CL, kGtEpiWarps * EPI::kWarpStaging>;
    constexpr bool F32 = OUT == kGt32;
    GtMaps m;
    bool ok = true;
    const uint64_t rows = uint64_t(g.M > 0 ? g.M : 1);
    if (MODE == kGmmDw) {
        // with no rows nothing is loaded; the maps still need an address
        const void* a = g.M > 0 ? g.a : g.out;
        const void* b = g.M > 0 ? g.b : g.out;
        ok = gt_map16(&m.a.whole, a, g.N, rows, 0, 64) && gt_map16(&m.b, b, g.K, rows, 0, 64);
        m.a.part = m.a.whole;
        ok = ok && gt_map(&m.out, F32 ? 4 : 2, g.out, uint64_t(g.K) * (F32 ? 4 : 2), g.N, g.E, 32);
    } else {
        const int red = MODE == kGmmFwd ? g.K : g.N;
        ok = gt_map16(&m.a.part, g.a, red, rows, 0, kGtBox) &&
             gt_map16(&m.a.whole, g.a, red, rows, 0, kGtRows) &&
             gt_map16(&m.b, g.b, g.K, g.N, g.E, MODE == kGmmFwd ? G::kCols : 64);
        m.out = m.b;
    }
    if (!ok) return cudaErrorInvalidValue;
    GtArgs a{};
    a.out = g.out;
    a.offsets = g.offsets;
    a.err = g.err;
    a.M = g.M;
    a.K = g.K;
    a.N = g.N;
    a.E = g.E;
    a.bf16 = g.dtype == STRATA_BF16;
    const size_t pitch = size_t(MODE == kGmmFwd ? g.N : g.K) * (F32 ? 4 : 2);
    a.vec = gt_vec(g.out, pitch);
    return gt_launch<k_gmm_tc<MODE, BN, OUT, CL, EPI>>(kGtThreads, cluster, grid, G::kDyn, s, m, a, epi);
}

template <int MODE, int BN, int CL, typename EPI>
cudaError_t gt_typed(const GmmArgs& g, int cluster, int grid, const EPI& epi, cudaStream_t s) {
    if constexpr (std::is_same<EPI, GtPlain>::value)
        if (g.out_dtype == STRATA_F32) return gt_run<MODE, BN, kGt32, CL>(g, cluster, grid, epi, s);
    // dw's reduction is a group's rows, which only the device knows
    if constexpr (MODE != kGmmDw)
        if ((MODE == kGmmFwd ? g.K : g.N) <= kGtDrain16 * kGtK)
            return gt_run<MODE, BN, kGt16, CL>(g, cluster, grid, epi, s);
    return gt_run<MODE, BN, kGt16Pieces, CL>(g, cluster, grid, epi, s);
}

// Which tiles.  dw: a CTA pair from 512 rows a group on average (us, 32
// experts of 1024 x 2048, single and pair, bf16: 44.4 51.6 at 256 rows, 57.6
// 52.0 at 384, 68.3 54.5 at 512, 115.2 88.5 at 1024; fp32: 56.9 68.1, 71.6 75.5,
// 84.7 74.5, 131.1 107.2).  The average is of the buffer's rows: 2048 rows of
// these groups in a buffer of 16384 take the pair, 39.5 instead of 28.2.
//
// Forward and dx: the shortest by a count of waves and stages.  A stage takes
// a CTA about 0.25 us with 128 columns, 0.385 with 256, a pair (256 rows, 256
// columns) 0.35, however few of its rows are live; blocks are what the groups
// need on average (a half-empty last one each).  Single with 256 columns
// against pair, forward, same experts: 27.5 30.3 at 64 rows a group, 37.3 31.9
// at 128, 46.1 40.7 at 256, 57.3 58.0 at 512, 100.7 90.5 at 1024; 16 rows of
// 16 experts: 16.5, 14.0 with 128 columns.  Where even 128 columns leave most
// SMs idle, a cluster of up to 8 CTAs splits the reduction (1.5 us to join).
template <int MODE, typename EPI>
cudaError_t gt_pick(const GmmArgs& g, const EPI& epi, cudaStream_t s) {
    const int sms = device_info().sms, pairs = sms >= 2 ? sms / 2 * 2 : 2;
    if constexpr (MODE == kGmmDw) {
        if (g.M / g.E >= 512) return gt_typed<MODE, 256, kGtPair>(g, 2, pairs, epi, s);
        return gt_typed<MODE, 256, 0>(g, 1, sms, epi, s);
    } else {
        const long long cols = MODE == kGmmFwd ? g.N : g.K;
        const int stages = ((MODE == kGmmFwd ? g.K : g.N) + kGtK - 1) / kGtK;
        const long long groups = g.M < g.E ? g.M : g.E;
        const long long nt128 = (cols + 127) / 128, nt256 = (cols + 255) / 256;
        auto blocks = [&](int rows) {
            const long long b = g.M / rows + groups / 2;
            return b > groups ? b : groups;
        };
        auto cost = [&](long long tiles, int workers, double stage) {
            return double((tiles + workers - 1) / workers) * stages * stage;
        };
        const double c128 = cost(blocks(128) * nt128, sms, 0.25);
        const double c256 = cost(blocks(128) * nt256, sms, 0.385);
        const double cpair = cost(blocks(256) * nt256, pairs / 2, 0.35);
        // the most tiles that the offsets can make, so that a cluster takes one
        const long long most = (groups + g.M / kGtRows) * nt128;
        for (int parts = 8; parts >= 2; parts /= 2) {
            // clusters of 8 do not fill every part of the GPU
            if (most * parts > (parts == 8 ? sms - 24 : sms) || stages < 4 * parts) continue;
            const double split = (stages + parts - 1) / parts * 0.25 + 1.5;
            if (split < c128 && split < c256 && split < cpair)
                return gt_typed<MODE, 128, kGtSplit>(g, parts, int(most) * parts, epi, s);
        }
        if (cpair < c128 && cpair < c256) return gt_typed<MODE, 256, kGtPair>(g, 2, pairs, epi, s);
        if (c128 < c256) return gt_typed<MODE, 128, 0>(g, 1, sms, epi, s);
        return gt_typed<MODE, 256, 0>(g, 1, sms, epi, s);
    }
}

}  // namespace

}  // namespace strata
