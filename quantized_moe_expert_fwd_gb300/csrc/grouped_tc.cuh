// grouped_tc.cuh -- what the tensor-core kernels of the grouped products
// share: the CTA's roles, bounded waits, output stores, tensor maps, launch.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "grouped.cuh"
#include "grouped.h"
#include "tc.cuh"

namespace strata {

constexpr int kGtThreads = 320;
constexpr int kGtEpiWarps = 8, kGtTmaWarp = 8, kGtMmaWarp = 9;
constexpr int kGtRows = 128;                    // tile rows
constexpr int kGtBox = 32;                      // rows of the smaller row box

// What the waits of a CTA share beside the workspace's error word: two words of
// shared memory, which a pair's CTAs keep alike.  stop is set once a wait has
// run out; the others then give up early.  (Not by the error word: a code
// latched by an earlier call, and not read yet, must not cut this call's waits
// short.)  halted: a bit for each CTA whose producer then issues nothing more.
struct GtStop {
    uint32_t stop, halted;
};
template <bool PAIR>
struct GtWaits {
    uint32_t* err;
    GtStop* s;
    __device__ __forceinline__ bool seen(const uint32_t* word, uint32_t value) const {
        return *reinterpret_cast<const volatile uint32_t*>(word) == value;
    }
    __device__ __forceinline__ void mark(uint32_t* word, uint32_t bit) const {
        if (PAIR) {
            or_cluster_u32(word, 0, bit);
            or_cluster_u32(word, 1, bit);
        } else {
            atomicOr(word, bit);
        }
    }
};

// Bounded wait (a poll lasts about 2 us, the limit 8 s; CLUSTER: sees what both
// CTAs of a pair did).  After one that ran out, the producers issue nothing
// more.  The MMA warp and the 4-bit kernel's scale warps (HOLD) go on once they
// have seen that: they hand stages back that may not have landed, and a second
// expected count in one phase would be undefined.  Without them the producers
// come to wait themselves, so their own limit is twice as long.  All but the
// producers run on to their end over values that nobody is to use: their
// arrivals only complete phases, and stay within the CTA's own buffers.  (A
// check a stage that leaves the MMA loop cost 5 %; a look at the words every 16
// polls instead of 256, up to 5 too.)  EARLY = false: to the limit in any case,
// for what has to be over before the CTA gives its memory back.
template <bool CLUSTER = false, bool HOLD = false, bool EARLY = true, bool PAIR>
__device__ __forceinline__ bool gt_wait(uint64_t* bar, uint32_t parity, const GtWaits<PAIR>& w,
                                        uint32_t site, uint32_t slot) {
    for (uint32_t i = 0; i < (HOLD ? 2 * kWaitLimit : kWaitLimit); ++i) {
        if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if (EARLY && (i & 255u) == 255u &&
            (HOLD ? w.seen(&w.s->halted, PAIR ? 3u : 1u) : w.seen(&w.s->stop, 1u)))
            return false;
    }
    w.mark(&w.s->stop, 1u);
    latch_timeout(w.err, site, slot, parity, 0);
    return false;
}
// About a millisecond, far more than a copy under way takes: for copies of a
// call whose waits ran out and that no barrier here reports.
__device__ __forceinline__ void gt_settle() {
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// A CTA's (or CTA pair's) tiles in order: column tile c (of nt) fastest, then row block m, and
// with MT row blocks an expert (dw) the expert e.  Steps of one tile a
// worker are added digit by digit: a 64-bit division a tile took longer than the
// tile's first copies.
template <bool EXPERTS>
struct GtIter {
    int c, m, e, nt, mt, dc, dm, de;
    __device__ __forceinline__ GtIter(int nt_, int mt_, int worker, int workers)
        : e(0), nt(nt_), mt(mt_), de(0) {
        c = worker % nt;
        m = worker / nt;
        dc = workers % nt;
        dm = workers / nt;
        if (EXPERTS) {
            e = m / mt;
            m %= mt;
            de = dm / mt;
            dm %= mt;
        }
    }
    __device__ __forceinline__ void next() {
        c += dc;
        m += dm;
        if (c >= nt) {
            c -= nt;
            ++m;
        }
        if (EXPERTS) {
            e += de;
            if (m >= mt) {
                m -= mt;
                ++e;
            }
        }
    }
};

// N consecutive columns of one output row from fp32 values; nv of them
// exist.  A lane writes whole 32-byte sectors where the rows are aligned
// for it (vec: the bytes that every row is aligned to: 32, 16 or 0).
__device__ __forceinline__ void gt_st8(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// WORDS words of a row whose pieces of 32 bytes are aligned; `have` bytes of
// them exist (a whole number of 16).
template <int WORDS>
__device__ __forceinline__ void gt_store_words(uint8_t* p, const uint32_t (&w)[WORDS], int have) {
    if (have >= WORDS * 4) {
#pragma unroll
        for (int i = 0; i < WORDS; i += 8) gt_st8(p + i * 4, w + i);
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4)
            if (i * 4 < have)
                *reinterpret_cast<uint4*>(p + i * 4) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}
// The same of rows aligned to 16 bytes only, from the warp's staging (17
// words a row): neighbouring lanes write a row's neighbouring 16 bytes.
template <int WORDS>
__device__ __forceinline__ void gt_store_staged(uint8_t* p, size_t pitch, int rows,
                                                const uint32_t* stage, int have) {
    constexpr int PER = WORDS / 4, STEP = 32 / PER;          // lanes a row, rows an instruction
    const int lane = threadIdx.x & 31, q = lane % PER;
    if (q * 16 >= have) return;
#pragma unroll
    for (int k = 0; k < 32 / STEP; ++k) {
        const int r = k * STEP + lane / PER;
        const uint32_t* s = stage + r * 17 + q * 4;
        if (r < rows)
            *reinterpret_cast<uint4*>(p + r * pitch + q * 16) = make_uint4(s[0], s[1], s[2], s[3]);
    }
}
__device__ __forceinline__ uint32_t gt_pack(float lo, float hi, int bf16) {
    uint32_t r;
    if (bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// N columns (nv of them exist) of a warp's 32 output rows, `rows` of them
// live, from each lane's fp32 values of its own row; `at` is the first row's
// place, `pitch` the row length.  Rows aligned to 32 bytes (vec) are written
// by their lanes, whole sectors each.  Others go through shared memory, so
// that neighbouring lanes write neighbouring columns: a lane a row wrote 2 or
// 16 bytes into each of 32 sectors at a time (118 columns of 3008 rows: 22 us,
// now 7; 1928 columns of 9056 rows: 23, now 19).
constexpr uint32_t kGtStoreWords = 32 * 17;               // a warp's staging
constexpr uint32_t kGtStoreBytes = kGtEpiWarps * kGtStoreWords * 4;
template <bool F32, int N>
__device__ __forceinline__ void gt_store(void* out, size_t at, size_t pitch, int rows,
                                         const float* v, int nv, int vec, int bf16,
                                         uint32_t* stage) {
    if (rows <= 0 || nv <= 0) return;
    const int lane = threadIdx.x & 31;
    if (F32) {
        float* p = static_cast<float*>(out) + at;
        if (vec == 32) {
            uint32_t w[N];
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = __float_as_uint(v[j]);
            if (lane < rows)
                gt_store_words(reinterpret_cast<uint8_t*>(p + lane * pitch), w, nv * 4);
            return;
        }
        // 16 columns at a time, two rows an instruction
        const int c = lane & 15;
#pragma unroll
        for (int h = 0; h < N; h += 16) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) stage[lane * 17 + j] = __float_as_uint(v[h + j]);
            __syncwarp();
            if (vec) {
                gt_store_staged<16>(reinterpret_cast<uint8_t*>(p + h), pitch * 4, rows, stage,
                                    (nv - h) * 4);
                continue;
            }
            float* o = p + size_t(lane >> 4) * pitch + h + c;
            const uint32_t* s = stage + (lane >> 4) * 17 + c;
#pragma unroll 4
            for (int r = lane >> 4; r < rows; r += 2, o += 2 * pitch, s += 2 * 17)
                if (h + c < nv) *o = __uint_as_float(*s);
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(out) + at;
        uint32_t w[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) w[j] = gt_pack(v[2 * j], v[2 * j + 1], bf16);
        if (vec == 32) {
            if (lane < rows)
                gt_store_words(reinterpret_cast<uint8_t*>(p + lane * pitch), w, nv * 2);
            return;
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < N / 2; ++j) stage[lane * 17 + j] = w[j];
        __syncwarp();
        if (vec) {
            gt_store_staged<N / 2>(reinterpret_cast<uint8_t*>(p), pitch * 2, rows, stage, nv * 2);
            return;
        }
        constexpr int STEP = 32 / N;                        // rows an instruction
        const int c = lane % N;
        const uint16_t* s = reinterpret_cast<const uint16_t*>(stage) + (lane / N) * 34 + c;
        uint16_t* o = p + size_t(lane / N) * pitch + c;
#pragma unroll 4
        for (int r = lane / N; r < rows; r += STEP, o += STEP * pitch, s += STEP * 34)
            if (c < nv) *o = *s;
    }
}

// ------------------------------------------------------------------- host
inline PFN_cuTensorMapEncodeTiled_v12000 gt_encode_fn() {
    static std::mutex mu;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (fn == nullptr) {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}


// A row-major array [z][rows][inner bytes] with the 128-byte swizzle; boxes
// of 128 bytes by box_rows rows.  z = 0: two dimensions.  esize: bytes of an
// element (1, 2 or 4), the unit of the inner coordinate.
inline bool gt_map(CUtensorMap* m, int esize, const void* base, uint64_t inner, uint64_t rows,
                   uint64_t z, uint32_t box_rows) {
    auto fn = gt_encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dim[3] = {inner / esize, rows, z};
    const cuuint64_t stride[2] = {inner, inner * rows};
    const cuuint32_t box[3] = {cuuint32_t(128 / esize), box_rows, 1}, one[3] = {1, 1, 1};
    const CUtensorMapDataType type = esize == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_UINT32;
    return fn(m, type, z ? 3 : 2, const_cast<void*>(base), dim, stride, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool gt_map16(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t z,
                     uint32_t box_rows) {
    return gt_map(m, 2, base, inner * 2, rows, z, box_rows);
}

// Boxes of 32 and of 128 rows of the row operand: a tile that is nearly whole
// takes the larger one, any other as many of the smaller as its rows need.
struct GtRowMaps {
    CUtensorMap part, whole;
};

inline int gt_vec(const void* out, size_t pitch) {
    const size_t mis = pitch | reinterpret_cast<uintptr_t>(out);
    return mis % 32 == 0 ? 32 : mis % 16 == 0 ? 16 : 0;
}

// `grid` CTAs in clusters of `cluster`, after the grids before them
// (programmatic dependent launch: the kernel's prologue overlaps their tail).
template <auto KERNEL, typename... A>
cudaError_t gt_launch(int threads, int cluster, int grid, size_t dyn, cudaStream_t s,
                      const A&... args) {
    // the shared memory limit, raised once per device (again where a launch is
    // refused: a device that was reset has forgotten it)
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    for (int k = 0; k < 2; ++k) {
        const bool known = dev < 64 && (raised.load(std::memory_order_relaxed) & bit) != 0;
        if (!known || k > 0) {
            e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, int(dyn));
            if (e != cudaSuccess) return e;
            raised.fetch_or(bit, std::memory_order_relaxed);
        }
        e = cudaLaunchKernelEx(&cfg, KERNEL, args...);
        if (e != cudaErrorInvalidValue || !known) break;
        cudaGetLastError();
    }
    return e;
}

}  // namespace strata
