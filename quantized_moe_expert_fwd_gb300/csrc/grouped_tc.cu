// grouped_tc.cu -- the grouped products on the tensor cores.
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
//
// fp32 outputs: the tensor cores truncate as they add (relative error 2e-6 at
// 2048 terms, growing with their number), so the accumulator is drained every
// 512 terms into fp32 registers of the epilogue, where it is added with
// rounding (5e-7 at any length).  16-bit outputs round away far more than
// that and take the whole reduction in one accumulator.
#include "grouped_tc.cuh"

namespace strata {

namespace {

constexpr int kGtK = 64;                        // reduction of a stage (128 bytes)
constexpr int kGtPromote = 8;                   // stages between drains of an fp32 output
constexpr uint32_t kGtABytes = kGtRows * 128;
constexpr uint32_t kGtSub = 64 * 128;           // a 64 x 64 MN-major sub-block

// dw writes a whole tile for every stage or two that it reads: it gives up a
// stage for the output's staging, a piece of 32 rows by 128 bytes an epilogue
// warp (two pieces a warp and a stage less: 16384 rows 196 us instead of 192,
// 65536 rows 215 instead of 202).
constexpr uint32_t kGtPiece = 32 * 128;
constexpr uint32_t kGtStaging = kGtEpiWarps * kGtPiece;

// A kernel's geometry.  PAIR: two CTAs make one tile of 256 rows by BN
// columns; each loads its 128 rows and half of the columns.
template <int MODE, int BN, bool PAIR>
struct Gt {
    static constexpr int kCols = PAIR ? BN / 2 : BN;             // B columns a CTA loads
    static constexpr uint32_t kBBytes = uint32_t(kCols) * 128u;
    static constexpr uint32_t kStage = kGtABytes + kBBytes;
    static constexpr uint32_t kStagingBytes = MODE == kGmmDw ? kGtStaging : 0u;
    static constexpr int kStages = int((212992u - kStagingBytes) / kStage);
    static constexpr size_t kDyn = size_t(kStages) * kStage + kStagingBytes + 1024;
    static constexpr int kBlock = PAIR ? 2 * kGtRows : kGtRows;  // rows of a tile
};

struct GtMaps {
    CUtensorMap a[kGtRows / kGtBox];            // by box height (dw: a[0] alone)
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

struct GtTile {
    int e, arow, rows, c0, stages, slot0, cnt;
    size_t orow;
};

// rank: the CTA's half of a pair's rows.
template <int MODE, int BN, bool PAIR>
__device__ __forceinline__ GtTile gt_tile(const GroupTable& t, const GtArgs& a,
                                          const GtIter<MODE == kGmmDw>& it, int rank) {
    constexpr int BLOCK = Gt<MODE, BN, PAIR>::kBlock;
    GtTile i;
    i.c0 = it.c * BN;
    if (MODE == kGmmDw) {
        i.e = it.e;
        i.arow = it.m * BLOCK + rank * kGtRows;
        i.rows = min(kGtRows, a.N - i.arow);
        i.slot0 = t.row[i.e];
        i.cnt = t.cnt[i.e];
        i.stages = (i.cnt + kGtK - 1) / kGtK;
        i.orow = size_t(i.e) * a.N + i.arow;
    } else {
        i.e = group_of_block(t, a.E, it.m);
        const int in = (it.m - t.pre[i.e]) * BLOCK + rank * kGtRows;
        i.arow = t.row[i.e] + in;
        i.rows = min(kGtRows, t.cnt[i.e] - in);
        i.slot0 = i.cnt = 0;
        i.stages = ((MODE == kGmmFwd ? a.K : a.N) + kGtK - 1) / kGtK;
        i.orow = size_t(i.arow);
    }
    return i;
}

// dw: the rows of stage ks that the last 16-row step takes from behind the
// group's end.
template <int MODE>
__device__ __forceinline__ int gt_dead(const GtTile& i, int ks) {
    return MODE == kGmmDw ? -min(kGtK, i.cnt - ks * kGtK) & 15 : 0;
}

template <int MODE, int BN, bool F32, bool PAIR>
__global__ void __launch_bounds__(kGtThreads, 1)
    k_gmm_tc(const __grid_constant__ GtMaps maps, GtArgs a) {
    using G = Gt<MODE, BN, PAIR>;
    constexpr int STAGES = G::kStages;
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
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, lane = tid & 31;
    const int wid = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform to the compiler
    const int rank = PAIR ? int(cluster_rank()) : 0;
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
        mbar_fence_init();
        tma_prefetch_map(&maps.b);
        tma_prefetch_map(&maps.a[0]);
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
        int(blockIdx.x) / (PAIR ? 2 : 1), int(gridDim.x) / (PAIR ? 2 : 1));
    const int blocks = t.pre[a.E];
    auto more = [&](const GtIter<MODE == kGmmDw>& it) {
        return MODE == kGmmDw ? it.e < a.E : it.m < blocks;
    };

    if (wid == kGtTmaWarp) {
        if (elect_one()) {
            uint32_t st = 0;
            for (auto it = first_tile; more(it); it.next()) {
                const GtTile i = gt_tile<MODE, BN, PAIR>(t, a, it, rank);
                // a pair always loads whole boxes, so that rank 0 knows the bytes of both
                const int nbox = PAIR || MODE == kGmmDw ? kGtRows / kGtBox
                                                        : (i.rows + kGtBox - 1) / kGtBox;
                const CUtensorMap* ma = &maps.a[MODE == kGmmDw ? 0 : nbox - 1];
                const int b0 = i.c0 + rank * G::kCols;
                const uint32_t bytes = uint32_t(nbox) * kGtBox * 128u + G::kBBytes;
                for (int ks = 0; ks < i.stages; ++ks, ++st) {
                    const uint32_t s = st % STAGES, round = st / STAGES;
                    if (round > 0) gt_wait(&empty[s], (round - 1) & 1, a.err, 50, s);
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
            // every copy has landed (a pair's: has been consumed) before the CTA exits
            for (uint32_t k = st > STAGES ? st - STAGES : 0; k < st; ++k)
                gt_wait(PAIR ? &empty[k % STAGES] : &full[k % STAGES], (k / STAGES) & 1, a.err, 51,
                        k % STAGES);
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
            const GtTile i = gt_tile<MODE, BN, PAIR>(t, a, it, rank);
            for (int ks = 0; ks < i.stages; ++ks, ++st) {
                const uint32_t s = st % STAGES;
                const bool first = F32 ? ks % kGtPromote == 0 : ks == 0;
                const bool last = ks == i.stages - 1 || (F32 && ks % kGtPromote == kGtPromote - 1);
                const uint32_t buf = acc & 1u;
                if (rank == 0 && first && acc >= 2)
                    gt_wait<PAIR>(&acc_empty[buf], ((acc >> 1) - 1) & 1, a.err, 52, buf);
                uint8_t* sa = base + s * STAGE;
                uint8_t* sb = sa + kGtABytes;
                const int dead = gt_dead<MODE>(i, ks);         // rows of the next group
                int steps = kGtK / 16;
                if (MODE == kGmmDw) steps = (min(kGtK, i.cnt - ks * kGtK) + 15) / 16;
                if (!PAIR) {
                    gt_wait(&full[s], (st / STAGES) & 1, a.err, 53, s);
                } else if (dead == 0) {
                    if (rank == 0) {
                        gt_wait(&both[s], (both_phase >> s) & 1u, a.err, 56, s);
                        both_phase ^= 1u << s;
                    }
                } else {
                    gt_wait(&full[s], (own_phase >> s) & 1u, a.err, 53, s);
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
                        if (rank == 0) gt_wait<true>(&fixed[s], (own_phase >> s) & 1u, a.err, 57, s);
                        else if (elect_one()) mbar_arrive_rank0(&fixed[s]);
                        own_phase ^= 1u << s;
                    } else {
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                }
                if (rank != 0) {
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
        // no product may still be writing the TMEM when it is freed
        if (rank == 0 && elect_one()) {
            if (PAIR) umma2_commit(&done);
            else umma_commit(&done);
        }
        __syncwarp();
        gt_wait(&done, 0, a.err, 54, 0);
    } else {
        constexpr int CH = BN / 64;              // 32-column pieces of a warp's half
        const int half = wid >> 2, r = (wid & 3) * 32 + lane;
        const uint32_t tl = tmem + (uint32_t((wid & 3) * 32) << 16) + uint32_t(half * (BN / 2));
        uint8_t* stage = base + STAGES * STAGE + wid * kGtPiece;            // dw
        uint32_t acc = 0;
        // dw: 128 bytes of each of the warp's 32 rows to memory by TMA, which
        // writes whole lines (32-byte stores of a lane a row took 1.7 times
        // as long); the lanes' 16-byte pieces are spread by the swizzle
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
            const GtTile i = gt_tile<MODE, BN, PAIR>(t, a, it, rank);
            const int c0 = i.c0 + half * (BN / 2);
            const size_t at = (i.orow + r) * size_t(cols) + c0;
            const bool live = r < i.rows;
            if (F32) {
                float sum[CH][32];
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
                for (int ks = 0; ks < i.stages; ks += kGtPromote, ++acc) {
                    const uint32_t buf = acc & 1u;
                    gt_wait(&acc_full[buf], (acc >> 1) & 1, a.err, 55, buf);
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        uint32_t v[32];
                        tmem_ld32(tl + buf * BN + c * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c][j] += __uint_as_float(v[j]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR) mbar_arrive_rank0(&acc_empty[buf]);
                        else mbar_arrive(&acc_empty[buf]);
                    }
                }
                if (MODE == kGmmDw) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        put(i, c0 + c * 32, reinterpret_cast<const uint32_t(&)[32]>(sum[c]));
                } else if (live) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        gt_store<true, 32>(a.out, at + c * 32, sum[c], cols - c0 - c * 32, a.vec, 0);
                }
            } else {
                const uint32_t buf = acc & 1u;
                if (i.stages > 0) {
                    gt_wait(&acc_full[buf], (acc >> 1) & 1, a.err, 55, buf);
                    tc_fence_after();
                }
                uint32_t w[32];                  // dw: 64 columns, packed
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint32_t v[32];
                    if (i.stages > 0) {
                        tmem_ld32(tl + buf * BN + c * 32, v);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
                    if (MODE == kGmmDw) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            w[16 * (c & 1) + j] = gt_pack(__uint_as_float(v[2 * j]),
                                                          __uint_as_float(v[2 * j + 1]), a.bf16);
                        if (c & 1) put(i, c0 + (c - 1) * 32, w);
                    } else if (live) {
                        gt_store<false, 32>(a.out, at + c * 32, reinterpret_cast<const float*>(v),
                                            cols - c0 - c * 32, a.vec, a.bf16);
                    }
                }
                if (i.stages > 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR) mbar_arrive_rank0(&acc_empty[buf]);
                        else mbar_arrive(&acc_empty[buf]);
                    }
                    ++acc;
                }
            }
        }
        if (MODE == kGmmDw && lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();            // the other CTA reads and signals no more
    tc_fence_after();
    if (wid == kGtMmaWarp) {
        if (PAIR) tmem_dealloc2(tmem, 2 * BN);
        else tmem_dealloc(tmem, 2 * BN);
    }
}

// ------------------------------------------------------------------- host
template <int MODE, int BN, bool F32, bool PAIR>
cudaError_t gt_run(const GmmArgs& g, cudaStream_t s) {
    GtMaps m;
    bool ok = true;
    const uint64_t rows = uint64_t(g.M > 0 ? g.M : 1);
    if (MODE == kGmmDw) {
        // with no rows nothing is loaded; the maps still need an address
        const void* a = g.M > 0 ? g.a : g.out;
        const void* b = g.M > 0 ? g.b : g.out;
        ok = gt_map16(&m.a[0], a, g.N, rows, 0, 64) && gt_map16(&m.b, b, g.K, rows, 0, 64);
        for (int i = 1; i < kGtRows / kGtBox; ++i) m.a[i] = m.a[0];
        ok = ok && gt_map(&m.out, F32 ? 4 : 2, g.out, uint64_t(g.K) * (F32 ? 4 : 2), g.N, g.E, 32);
    } else {
        const int red = MODE == kGmmFwd ? g.K : g.N;
        for (int i = 0; i < kGtRows / kGtBox; ++i)
            ok = ok && gt_map16(&m.a[i], g.a, red, rows, 0, kGtBox * (i + 1));
        ok = ok && gt_map16(&m.b, g.b, g.K, g.N, g.E, MODE == kGmmFwd ? Gt<MODE, BN, PAIR>::kCols : 64);
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
    return gt_launch(k_gmm_tc<MODE, BN, F32, PAIR>, kGtThreads, PAIR ? 2 : 1,
                     Gt<MODE, BN, PAIR>::kDyn, s, m, a);
}

template <int MODE, int BN, bool PAIR>
cudaError_t gt_typed(const GmmArgs& g, cudaStream_t s) {
    return g.out_dtype == STRATA_F32 ? gt_run<MODE, BN, true, PAIR>(g, s)
                                     : gt_run<MODE, BN, false, PAIR>(g, s);
}

// Rows a group, on average, from which a CTA pair makes the tiles: half of the
// column operand's traffic, but tiles of 256 rows.  Single against pair, us,
// 32 experts of 1024 x 2048 in bf16:
//   rows a group    128        256        512        1024
//   forward     37.3 31.9  46.1 40.7  57.3 58.0  100.7  90.5
//   dx          31.4 31.3  39.5 36.5  58.2 56.0  101.0  94.6
//   dw          36.8 46.0  51.4 55.8  77.2 74.1  124.7 107.2
// (16384 x 4096 x 4096 in one group: 306 and 281, the library's product 270).
constexpr int gt_pair_rows(int mode) {
    return mode == kGmmFwd ? 128 : mode == kGmmDx ? 256 : 512;
}

template <int MODE>
cudaError_t gt_pick(const GmmArgs& g, cudaStream_t s) {
    // 256 columns a tile halve the row operand's traffic and the stages; 128
    // where twice the tiles still run side by side (16 rows of 16 experts of
    // 1024 x 2048: 14.0 us against 16.5; 32 rows: 24.9 against 24.1)
    const int cols = MODE == kGmmFwd ? g.N : g.K;
    const long long blocks = (g.M < g.E ? g.M : g.E) + g.M / kGtRows;
    if (g.M / g.E >= gt_pair_rows(MODE)) return gt_typed<MODE, 256, true>(g, s);
    if (MODE == kGmmDw) return gt_typed<MODE, 256, false>(g, s);
    if (2 * blocks * ((cols + 255) / 256) <= device_info().sms)
        return gt_typed<MODE, 128, false>(g, s);
    return gt_typed<MODE, 256, false>(g, s);
}

}  // namespace

// The tensor maps need rows of a multiple of 16 bytes.
bool grouped_tc_takes(GroupedMode mode, const GmmArgs& g) {
    return g.K % 8 == 0 && (mode == kGmmFwd || g.N % 8 == 0);
}

cudaError_t launch_grouped_tc(GroupedMode mode, const GmmArgs& g, cudaStream_t s) {
    switch (mode) {
        case kGmmFwd: return gt_pick<kGmmFwd>(g, s);
        case kGmmDx: return gt_pick<kGmmDx>(g, s);
        default: return gt_pick<kGmmDw>(g, s);
    }
}

}  // namespace strata
