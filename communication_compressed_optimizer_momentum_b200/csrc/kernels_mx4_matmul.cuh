// kernels_mx4_matmul.cuh -- products of two matrices in microscaled 4-bit floating point for B200
// (sm_100a): on the tensor cores, and without them for few rows.
#pragma once

#include <cuda.h>

#include "kernels_mx4.cuh"

namespace onebit {

// ------------------------------------------------------------------------------------------
// the product: out[i][j] = sum_k a[i][k] b[j][k]
//
// One thread block takes 128 columns of out (rows of b) by TM rows of out (rows of a). b's rows are the
// 128 lanes of the accumulator in tensor memory, so that a warp's stores of one row of out are
// consecutive whatever its strides are, and so that few rows of a (one token) take a narrow
// instruction rather than an empty one. A stage is 256 columns of both operands (128 bytes of a row,
// one 128-byte swizzle atom) with their exponents, four instructions of 64 columns.
//
// PAIR: two thread blocks of a cluster share a tile of 256 columns by 256 rows of out: each loads its
// 128 rows of b and half of the rows of a, and one instruction of the first block multiplies in both.
// That halves what each reads of a. The codes of both count on one barrier of the first block, which the
// warp that issues the products waits on; the exponents count in each block, whose warps store them.
//
// Warps: 0 loads (TMA), 1 issues the products, 2 to 9 write out (two for each quarter of the lanes), 10
// to 13 move the exponents from shared to tensor memory (each its quarter of the lanes; every quarter
// holds all of them). The tensor cores' own copies (tcgen05.cp) wait for the products before them and
// hold up those behind: 75 clocks an atom, six for every four products.
//
// 8192 x 8192 x 8192 to bf16 takes 166 us alone, 176 to 183 as one of 20 in a row, 210 after seconds of
// them: the tensor pipe is busy 85% of the time, at the clock that the power cap leaves (1.52 GHz). Short
// common axes are bound by loads and results sharing the path to L2 (8192 x 6400 from 1600 columns: 41 us,
// up to 54 in programs whose memory lies otherwise; 30 without storing), small products by their launch.

constexpr int kMmThreads = 448;
constexpr int kOutWarps = 8;              // write out
constexpr int kMmLanes = 128;             // rows of b in a block's part of a tile
constexpr int kStageCols = 256;
constexpr uint32_t kMmTimeout = 1u;
constexpr uint64_t kMmWaitNs = 20ull * 1000 * 1000 * 1000;   // the longest tile takes a second
constexpr int kOutBytes = 2048;           // written out at a time: 32 columns of out by 32 rows (bf16)
constexpr int kOutRows32 = 16;            // ... or by 16 (fp32)

__device__ uint32_t g_mx4_status;

// Whether phase `parity` of the barrier is over, seen without ordering memory, for arrivals from all of a
// cluster.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// Wait for phase `parity` of the barrier, giving up after `limit` ns (a long common axis keeps the warps
// that write out waiting for a good while: a number of polls would not say how long; 256 polls take 1 ms
// where nothing comes). The loops stay loops: unrolled, a layer's three passes take 1 us more.
// PAIR: arrivals come from the other block too (pair_arrive).
template <bool PAIR = false>
__device__ __forceinline__ bool mm_wait(uint64_t* bar, uint32_t parity, uint64_t limit) {
    const auto there = [&] {
        return PAIR ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
    };
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (there()) return true;
    uint64_t start, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(start));
    do {
#pragma unroll 1
        for (int i = 0; i < 256; ++i)
            if (there()) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    } while (now - start < limit);
    return false;
}

// The same for a warp that runs together: all of its lanes wait, and all give up if one does.
template <bool PAIR = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit) {
    return __all_sync(kFull, mm_wait<PAIR>(bar, parity, limit));
}

template <int TM, bool PAIR, bool SPLIT>
struct MmTile {
    static constexpr int kGroup = PAIR ? 2 : 1;
    static constexpr int kARows = TM / kGroup;                // rows of a that a block loads
    static constexpr int kHalves = TM > 128 ? 2 : 1;          // atoms of a's exponents across
    static constexpr int kB = kMmLanes * 128, kA = kARows * 128;  // bytes of codes in a stage
    static constexpr int kSB = 2 * kAtomBytes, kSA = 2 * kHalves * kAtomBytes;
    static constexpr int kStage = kB + kA + kSB + kSA;
    // Behind the stages: what is written out (a buffer for each warp), or the sums of a split tile from
    // the other blocks, [block][its rows][128].
    static constexpr int kParts = SPLIT ? (TM + 8) * kMmLanes * 4 : kOutWarps * kOutBytes;
    static constexpr int kBarriers = 512;
    static constexpr int kMost = (227 * 1024 - kBarriers - kParts) / kStage;
    static constexpr int kStages = kMost < 8 ? kMost : 8;
    static constexpr int kSmem = kStages * kStage + kParts + kBarriers;
    // Tensor memory: two accumulators and the exponents of as many stages as there are. Two of 256
    // columns leave no room: they overlap by 96 columns, which are read first, and four stages'
    // exponents are kept.
    static constexpr int kExpBuffers = TM == 256 ? 4 : kStages;
    static_assert(kStages >= kExpBuffers, "the exponents' buffers are freed with the stages");
    static constexpr int kOverlap = TM == 256 ? 96 : 0;
    static constexpr int kSecond = TM - kOverlap;
    static constexpr int kExp = kSecond + TM;
    static constexpr int kExpCols = 8 + 8 * kHalves;
    static constexpr int kNeed = kExp + kExpBuffers * kExpCols;
    static constexpr int kColumns = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static_assert(kNeed <= 512, "tensor memory");
    static constexpr int kChunk = TM <= 32 ? 16 : 32;         // columns taken out at a time
};

struct Mx4Maps {
    CUtensorMap a, b, sa, sb;  // codes and exponents
    CUtensorMap out;           // where Mx4MatmulArgs::tma
};

struct Mx4MatmulArgs {
    void* out;
    int64_t ld;
    int32_t m, n;              // rows and columns of out
    int32_t steps;             // products of 64 columns
    int32_t stages;            // of 256 columns
    int32_t tiles_m, tiles_n;
    int32_t accumulate;
    int32_t tma;               // out's address and rows are aligned to 16 bytes
    uint64_t wait_ns;          // after which a wait gives up
};

__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, int x, int y,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// The same for a pair, counted on a barrier of either block (`bar`: its address for the cluster).
__device__ __forceinline__ void tma_tile_pair(void* dst, const CUtensorMap* map, int x, int y,
                                              uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The barrier (of both blocks of a pair) completes when the products that this thread has issued so
// far are done.
template <bool PAIR>
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
            "[%0], %1;" ::"r"(smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(smem_addr(bar))
                     : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tc_product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sa, uint32_t sb, bool add) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
            "[%5], p;\n}\n"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
            "[%5], p;\n}\n"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
            : "memory");
}

// Shared memory descriptor: rows of 128 bytes in 128-byte swizzle atoms of eight (1024 bytes apart).
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | 1ull << 16 | (uint64_t)(1024 >> 4) << 32 |
           1ull << 46 | 2ull << 61;
}

// Both operands 4-bit (E2M1), exponents as powers of two, fp32 sums; half: which blocks of the
// exponents' words.
template <int TM, bool PAIR>
__device__ __forceinline__ uint32_t product_desc(uint32_t half) {
    return (2 * half) << 4 | 1u << 7 | 1u << 10 | (uint32_t)(TM / 8) << 17 | 1u << 23 |
           (uint32_t)(kMmLanes * (PAIR ? 2 : 1) / 16) << 24 | (2 * half) << 29;
}

// N columns of the warp's 32 lanes, a lane each: v[j] is column j.
template <int N>
__device__ __forceinline__ void tc_load(uint32_t addr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    if constexpr (N == 32)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                     "%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
                     "%31}, [%32];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                       "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                       "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                       "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
                       "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                     "%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                       "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(addr)
                     : "memory");
}
// N columns of 16 lanes as matrices of 8 x 8: v[4 i + 2 h + e] is lane 8 h + l / 4, column
// 8 i + 2 (l % 4) + e in the warp's lane l.
template <int N>
__device__ __forceinline__ void tc_load_matrices(uint32_t addr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    if constexpr (N == 32)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                     "%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                       "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "r"(addr)
                     : "memory");
}
// What has been loaded is there (the values pass through, so that no use moves before this).
template <int N>
__device__ __forceinline__ void tc_load_wait(float* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
// Eight columns of tensor memory, a word a lane each.
__device__ __forceinline__ void tc_store8(uint32_t addr, const uint4& a, const uint4& b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
                 "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address, for the cluster, of this block's `addr` in the block `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t p;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
    return p;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Arrive on a barrier of a pair's first block, which issues the products of both. Relaxed, at the
// cluster's scope: no memory is ordered by the arrival and by the wait for it themselves (with a release
// at this scope a warp stands still for 1000 clocks: 8192^3 takes 423 us, without 240; one warp that
// passes the others' arrivals on with a release: 400, where 180 are reached without).
// - Tensor memory (the exponents that are stored, the accumulators that are read) is ordered by the
//   tensor cores' own fences: the operation and its wait, tcgen05.fence::before_thread_sync, a relaxed
//   arrival; a relaxed wait, tcgen05.fence::after_thread_sync, the product. PTX gives this pattern.
// - The codes that the second block copies count on a barrier of the first, where the thread that issues
//   the products waits for them itself.
template <bool PAIR>
__device__ __forceinline__ void pair_arrive(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         cluster_addr(smem_addr(bar), 0))
                     : "memory");
    else
        mbar_arrive(bar);
}
// One lane of a warp that runs together: the compiler keeps what such a branch's instructions take in
// uniform registers, which a branch on the lane's number does not let it (200 clocks a product, so 128).
__device__ __forceinline__ bool elect() {
    uint32_t yes;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(yes));
    return yes != 0;
}

// What a warp writes out: a buffer in shared memory, and where it goes.
struct OutWarp {
    const CUtensorMap* map;
    uint8_t* buf;              // kOutBytes
    int n0;                    // the warp's first column of out
    int lane;
};

// The buffer, once the copy out of it is over.
__device__ __forceinline__ uint8_t* out_buffer(const OutWarp& w) {
    if (w.lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    return w.buf;
}
// Copy the buffer out, or add it, its first row being `row`; the map leaves out what lies behind the
// edges. Nobody else touches these values: there is one order of adding.
template <bool ADD>
__device__ __forceinline__ void out_copy(const OutWarp& w, int row) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (w.lane == 0) {
        if constexpr (ADD)
            asm volatile(
                "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], "
                "[%3];" ::"l"(w.map),
                "r"(w.n0), "r"(row), "r"(smem_addr(w.buf))
                : "memory");
        else
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                    w.map),
                "r"(w.n0), "r"(row), "r"(smem_addr(w.buf))
                : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// A chunk of N columns of the accumulator, from tensor memory to registers. bf16: as matrices, which
// stmatrix transposes on their way to shared memory.
template <int N, typename OT>
__device__ __forceinline__ void take_chunk(uint32_t addr, float* v) {
    if constexpr (sizeof(OT) == 4) {
        tc_load<N>(addr, v);
    } else {
        tc_load_matrices<N>(addr, v);
        tc_load_matrices<N>(addr + (16u << 16), v + N / 2);
    }
}

// Write a chunk out: rows row .. row + N - 1 of out, of which `rows` (or more) are there. The values
// go through shared memory and by TMA, which wants aligned rows; else element by element. (bf16 from
// 1600 columns, 8192 x 6400: two bytes a lane by plain stores 145 us; lanes exchanging values until
// each has eight columns of a row 61; by TMA 41. Rows that TMA does not take still go by two bytes a lane,
// out of shared memory: 8192 x 6401 92 us.)
template <int N, typename OT>
__device__ __forceinline__ void put_chunk(const Mx4MatmulArgs& p, OutWarp& w, float* v, int row,
                                          int rows) {
    const int lane = w.lane;
    if (rows <= 0 || w.n0 >= p.n) return;
    if constexpr (sizeof(OT) == 4) {
        float* const out = static_cast<float*>(p.out) + (int64_t)row * p.ld + w.n0 + lane;
        const bool in = w.n0 + lane < p.n;
#pragma unroll
        for (int h = 0; h < N; h += kOutRows32) {
            if (h >= rows) break;
            if (p.tma) {
                float* buf = reinterpret_cast<float*>(out_buffer(w));
#pragma unroll
                for (int j = 0; j < kOutRows32; ++j) buf[j * 32 + lane] = v[h + j];
                if (p.accumulate)
                    out_copy<true>(w, row + h);
                else
                    out_copy<false>(w, row + h);
            } else {
                float o[kOutRows32];
#pragma unroll
                for (int j = 0; j < kOutRows32; ++j)
                    o[j] = p.accumulate && in && h + j < rows ? out[(h + j) * p.ld] : 0.0f;
#pragma unroll
                for (int j = 0; j < kOutRows32; ++j)
                    if (in && h + j < rows)
                        out[(h + j) * p.ld] = p.accumulate ? o[j] + v[h + j] : v[h + j];
            }
        }
    } else {
        uint8_t* buf = out_buffer(w);
        // matrix g of a store: columns 8 g .. 8 g + 7 of out, 16 bytes of a row of 64; the 16-byte
        // pieces of a row are swapped as the map's 64-byte swizzle has them
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            uint32_t x[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float* q = v + (g >> 1) * (N / 2) + 4 * i + 2 * (g & 1);
                const __nv_bfloat162 h = __floats2bfloat162_rn(q[0], q[1]);
                x[g] = *reinterpret_cast<const uint32_t*>(&h);
            }
            const int r = 8 * i + (lane & 7);
            const uint32_t at = smem_addr(buf) + r * 64 + (((lane >> 3) ^ (r >> 1)) & 3) * 16;
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                             at),
                         "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
        }
        if (p.tma) {
            out_copy<false>(w, row);
        } else {
            __syncwarp();
            uint16_t* out = static_cast<uint16_t*>(p.out) + (int64_t)row * p.ld + w.n0 + lane;
            if (w.n0 + lane < p.n)
                for (int r = 0; r < N && r < rows; ++r)
                    out[r * p.ld] = *reinterpret_cast<const uint16_t*>(
                        buf + r * 64 + (((lane >> 3) ^ (r >> 1)) & 3) * 16 + (lane & 7) * 2);
            __syncwarp();
        }
    }
}

// SPLIT: a cluster of thread blocks shares one tile, each with a part of the common axis; every block
// sends its sums to the block that adds up their rows, which does so in the blocks' order. Otherwise
// a block (or a pair) walks over tiles, and the products of one tile run while the last one is
// written out.
template <int TM, bool PAIR, typename OT, bool SPLIT>
__global__ void __launch_bounds__(kMmThreads, 1)
k_mx4_matmul(const __grid_constant__ Mx4Maps maps, const Mx4MatmulArgs p) {
    static_assert(!(PAIR && SPLIT), "one or the other");
    using S = MmTile<TM, PAIR, SPLIT>;
    extern __shared__ __align__(1024) uint8_t mm_smem[];
    uint8_t* const sm = mm_smem;
    float* const parts = reinterpret_cast<float*>(sm + S::kStages * S::kStage);
    uint64_t* const full = reinterpret_cast<uint64_t*>(sm + S::kStages * S::kStage + S::kParts);
    uint64_t* const ready = full + S::kStages;      // ... and the exponents are in tensor memory
    uint64_t* const empty = ready + S::kStages;
    uint64_t* const codes = empty + S::kStages;     // PAIR: both blocks' codes, in the first one's
    uint64_t* const done = codes + S::kStages;      // [2] an accumulator is complete
    uint64_t* const drained = done + 2;             // [2] ... and read as far as the next needs
    uint64_t* const last = drained + 2;
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(last + 1);
    const int warp = (int)__shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(ready + i, 4 * S::kGroup);
            mbar_init(empty + i, 1);
            mbar_init(codes + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(done + i, 1);
            mbar_init(drained + i, kOutWarps * S::kGroup);
        }
        mbar_init(last, 1);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_addr(tmem_at)),
                         "r"(S::kColumns)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_addr(tmem_at)),
                         "r"(S::kColumns)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
        tc_fence_before();
    }
    __syncthreads();
    if constexpr (PAIR || SPLIT) {
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    after_what_is_ahead();

    const int rank = PAIR || SPLIT ? (int)cluster_rank() : 0;
    const int tiles = p.tiles_m * p.tiles_n;
    const int nsplit = SPLIT ? (int)gridDim.x / tiles : 1;
    const int first = SPLIT ? (int)blockIdx.x / nsplit : (int)blockIdx.x / S::kGroup;
    const int hop = SPLIT ? tiles : (int)gridDim.x / S::kGroup;
    const int k0 = SPLIT ? (int)((int64_t)p.stages * rank / nsplit) : 0;
    const int k1 = SPLIT ? (int)((int64_t)p.stages * (rank + 1) / nsplit) : p.stages;
    const int bank = PAIR ? rank : 0;               // which of the tile's rows of b
    // Bands of 16 (8) tiles along b's rows, so that the tiles that run together share their operands
    // in L2.
    constexpr int kBand = 16 / S::kGroup;
    const auto place = [&](int t, int& tm, int& tn) {
        const int band = t / (kBand * p.tiles_m);
        const int wide = min(kBand, p.tiles_n - band * kBand);
        const int r = t - band * kBand * p.tiles_m;
        tm = r / wide;
        tn = band * kBand + r % wide;
    };
    // A warp that gives up stops, and those that depend on it do likewise, each for itself: what is
    // in flight is waited for at the end by the warp that has started it, whether it has given up or
    // not, and with a limit of its own, since copies and products that have been issued do end.
    bool ok = true;

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0;
        int64_t filled = 0;
        for (int t = first; t < tiles && ok; t += hop) {
            int tm, tn;
            place(t, tm, tn);
            const int arow = tm * TM / kAtomRows, brow = tn * S::kGroup + bank;
            for (int k = k0; k < k1; ++k) {
                if (!(ok = warp_wait(empty + stage, phase ^ 1, p.wait_ns))) break;
                uint8_t* s = sm + stage * S::kStage;
                if (elect()) {
                    // A pair's codes count where they are waited for. (The second block's may come
                    // before the first has said how many bytes to expect, but not in another phase: that
                    // stage's last products have waited for all of the last phase.)
                    const int arow0 = tm * TM + bank * S::kARows;
                    if constexpr (PAIR) {
                        const uint32_t bar = cluster_addr(smem_addr(codes + stage), 0);
                        if (bank == 0) mbar_arrive_expect_tx(codes + stage, 2 * (S::kB + S::kA));
                        tma_tile_pair(s, &maps.b, k * 128, brow * kMmLanes, bar);
                        tma_tile_pair(s + S::kB, &maps.a, k * 128, arow0, bar);
                        mbar_arrive_expect_tx(full + stage, S::kSB + S::kSA);
                    } else {
                        mbar_arrive_expect_tx(full + stage, S::kStage);
                        tma_tile(s, &maps.b, k * 128, brow * kMmLanes, full + stage);
                        tma_tile(s + S::kB, &maps.a, k * 128, arow0, full + stage);
                    }
                    tma_tile(s + S::kB + S::kA, &maps.sb, k * 256, brow, full + stage);
                    tma_tile(s + S::kB + S::kA + S::kSB, &maps.sa, k * 256, arow, full + stage);
                }
                __syncwarp();
                ++filled;
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (lane == 0) {         // leave no copy in flight behind
            for (int64_t f = filled > S::kStages ? filled - S::kStages : 0; f < filled; ++f) {
                const int at = (int)(f % S::kStages);
                const uint32_t parity = (uint32_t)(f / S::kStages) & 1;
                ok = mm_wait(full + at, parity, kMmWaitNs) && ok;
                // A pair's codes: the products that read them are done, or a wait of this warp has run
                // out since they were queued (a copy takes microseconds, a wait a millisecond at least).
                if (PAIR && ok) ok = mm_wait(empty + at, parity, p.wait_ns);
            }
            // ... nor an arrival from a pair's other block, which may wait as long for one thing more
            if (PAIR && bank == 1) ok = mm_wait(last, 0, 4 * kMmWaitNs) && ok;
            if (!ok) atomicOr(&g_mx4_status, kMmTimeout);
        }
        __syncwarp();
    } else if (warp == 1 && bank == 0) {
        int stage = 0, c = 0;
        uint32_t phase = 0;
        int i = 0;
        for (int t = first; t < tiles && ok; t += hop, ++i) {
            int tm, tn;
            place(t, tm, tn);
            const uint32_t d = tmem + (uint32_t)(i & 1) * S::kSecond;
            const int before = S::kOverlap > 0 ? i - 1 : i - 2;  // the tile that has to be read first
            if (before >= 0 &&
                !(ok = warp_wait<PAIR>(drained + (before & 1), (uint32_t)(before >> 1) & 1, p.wait_ns)))
                break;
            tc_fence_after();
            for (int k = k0; k < k1; ++k, ++c) {
                // (the codes come before the exponents are stored: the second wait is the longer one)
                if (PAIR && !(ok = warp_wait(codes + stage, phase, p.wait_ns))) break;
                if (!(ok = warp_wait<PAIR>(ready + stage, phase, p.wait_ns))) break;
                tc_fence_after();
                const uint32_t s = smem_addr(sm + stage * S::kStage);
                const uint32_t eb = tmem + S::kExp + (c % S::kExpBuffers) * S::kExpCols, ea = eb + 8;
                const int steps = min(4, p.steps - 4 * k);
                if (elect()) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (q < steps)
                            tc_product<PAIR>(d, tile_desc(s) + 2 * q, tile_desc(s + S::kB) + 2 * q,
                                             product_desc<TM, PAIR>(q & 1), eb + 4 * (q >> 1),
                                             ea + 4 * S::kHalves * (q >> 1), k > k0 || q > 0);
                    tc_commit<PAIR>(empty + stage);
                }
                __syncwarp();
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (ok && elect()) tc_commit<PAIR>(done + (i & 1));
            __syncwarp();
        }
        if (elect()) {           // (the lane that issued them)
            tc_commit<PAIR>(last);
            ok = mm_wait(last, 0, kMmWaitNs) && ok;
            if (!ok) atomicOr(&g_mx4_status, kMmTimeout);
        }
    } else if (warp >= 2 && warp < 2 + kOutWarps) {
        const int quad = warp & 3, half = (warp - 2) >> 2;
        OutWarp w{&maps.out, reinterpret_cast<uint8_t*>(parts) + (warp - 2) * kOutBytes, 0, lane};
        int i = 0;
        for (int t = first; t < tiles && ok; t += hop, ++i) {
            int tm, tn;
            place(t, tm, tn);
            const int buf = i & 1;
            const uint32_t d = tmem + buf * S::kSecond + ((uint32_t)(quad * 32) << 16);
            const int64_t m0 = (int64_t)tm * TM;
            const int rows = (int)min((int64_t)TM, p.m - m0);
            w.n0 = (tn * S::kGroup + bank) * kMmLanes + quad * 32;
            constexpr int kC = S::kChunk;
            if (!(ok = warp_wait(done + buf, (uint32_t)(i >> 1) & 1, p.wait_ns))) break;
            tc_fence_after();
            const auto read_done = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pair_arrive<PAIR>(drained + buf);
            };
            if constexpr (SPLIT) {
                // lane j: the block that adds row j up, and this block's place there
                static_assert(!SPLIT || TM <= 32, "a row a lane");
                uint32_t to_row = 0;
                if (lane < rows) {
                    const int to = ((lane + 1) * nsplit - 1) / rows;
                    const int lo = rows * to / nsplit, count = rows * (to + 1) / nsplit - lo;
                    to_row = cluster_addr(smem_addr(parts + (rank * count + lane - lo) * kMmLanes),
                                          (uint32_t)to);
                }
                float v[kC];
                const int j0 = half * kC;
                if (j0 < TM) {
                    __syncwarp();
                    tc_load<kC>(d + j0, v);
                    tc_load_wait<kC>(v);
#pragma unroll
                    for (int j = 0; j < kC; ++j) {
                        const uint32_t at = __shfl_sync(kFull, to_row, j0 + j);
                        if (j0 + j < rows) cluster_store(at + (quad * 32 + lane) * 4, v[j]);
                    }
                }
            } else if constexpr (S::kOverlap > 0) {
                // what the accumulators share first: the last 96 columns of the first, the first of the
                // second, two chunks of the three for one warp; of the other five two as well
                static_assert(TM == 256 && S::kOverlap == 96 && kC == 32, "the warps' shares");
                const int at = (buf == 0 ? TM - 96 : 0) + (half == 0 ? 0 : 64);
                const int rest = (buf == 0 ? 0 : 96) + (half == 0 ? 0 : 64);
                const int to = rest + (half == 0 ? 64 : 96);
                float v[2 * kC];
                __syncwarp();
                take_chunk<kC, OT>(d + at, v);
                if (half == 0) take_chunk<kC, OT>(d + at + kC, v + kC);
                tc_load_wait<2 * kC>(v);
                read_done();
                put_chunk<kC, OT>(p, w, v, (int)m0 + at, rows - at);
                if (half == 0) put_chunk<kC, OT>(p, w, v + kC, (int)m0 + at + kC, rows - at - kC);
#pragma unroll 1
                for (int j0 = rest; j0 < to && j0 < rows; j0 += kC) {
                    __syncwarp();
                    take_chunk<kC, OT>(d + j0, v);
                    tc_load_wait<kC>(v);
                    put_chunk<kC, OT>(p, w, v, (int)m0 + j0, rows - j0);
                }
            } else {
                if (half * kC >= TM) read_done();
#pragma unroll 1
                for (int j0 = half * kC; j0 < TM; j0 += 2 * kC) {
                    float v[kC];
                    __syncwarp();
                    take_chunk<kC, OT>(d + j0, v);
                    tc_load_wait<kC>(v);
                    if (j0 + 2 * kC >= TM) read_done();
                    put_chunk<kC, OT>(p, w, v, (int)m0 + j0, rows - j0);
                }
            }
        }
        if (!SPLIT && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok && lane == 0) atomicOr(&g_mx4_status, kMmTimeout);
    } else if (warp >= 2 + kOutWarps) {
        int stage = 0, c = 0;
        uint32_t phase = 0;
        for (int t = first; t < tiles && ok; t += hop) {
            int tm, tn;
            place(t, tm, tn);
            // narrow tiles: the word of the tile's first rows (32 of the atom's 128 a word) comes first,
            // since the tensor cores take exponents from even columns on only
            const int sub = TM < kAtomRows ? tm * TM % kAtomRows / 32 : 0;
            for (int k = k0; k < k1; ++k, ++c) {
                if (!(ok = warp_wait(full + stage, phase, p.wait_ns))) break;
                const uint4* e = reinterpret_cast<const uint4*>(sm + stage * S::kStage + S::kB + S::kA) +
                                 lane;
                const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + S::kExp +
                                    (c % S::kExpBuffers) * S::kExpCols;
                uint4 w[2 + 2 * S::kHalves];
#pragma unroll
                for (int u = 0; u < 2 + 2 * S::kHalves; ++u) w[u] = e[u * (kAtomBytes / 16)];
                if constexpr (TM < kAtomRows) {
#pragma unroll
                    for (int u = 2; u < 4; ++u) {
                        const uint4 x = w[u];
                        w[u].x = sub == 0 ? x.x : sub == 1 ? x.y : sub == 2 ? x.z : x.w;
                        w[u].y = sub == 0 ? x.y : sub == 2 ? x.w : 0u;   // rows 32 to 63, if any
                    }
                }
                // the products that read this buffer before are done (with as many as stages, those of
                // the stage itself, for which its loads have waited)
                const int b = c - S::kExpBuffers;
                if (S::kExpBuffers < S::kStages && b >= 0 &&
                    !(ok = warp_wait(empty + b % S::kStages, (uint32_t)(b / S::kStages) & 1, p.wait_ns)))
                    break;
                __syncwarp();
                tc_fence_after();
                tc_store8(at, w[0], w[1]);
                if constexpr (S::kHalves == 1) {
                    tc_store8(at + 8, w[2], w[3]);
                } else {  // both halves of the first 128 columns, then of the second
                    tc_store8(at + 8, w[2], w[4]);
                    tc_store8(at + 16, w[3], w[5]);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pair_arrive<PAIR>(ready + stage);
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) atomicOr(&g_mx4_status, kMmTimeout);
    }
    __syncwarp();
    if constexpr (PAIR || SPLIT) {
        cluster_arrive();
        cluster_wait();
    }
    if constexpr (SPLIT) {
        int tm, tn;
        place(first, tm, tn);
        const int64_t m0 = (int64_t)tm * TM;
        const int rows = (int)min((int64_t)TM, p.m - m0);
        const int lo = rows * rank / nsplit, count = rows * (rank + 1) / nsplit - lo;
        for (int x = threadIdx.x; x < count * kMmLanes; x += kMmThreads) {
            float v = parts[x];
            for (int r = 1; r < nsplit; ++r) v += parts[r * count * kMmLanes + x];
            const int n = tn * kMmLanes + x % kMmLanes;
            OT* o = static_cast<OT*>(p.out) + (m0 + lo + x / kMmLanes) * p.ld + n;
            if (n < p.n) {
                if (sizeof(OT) == 4 && p.accumulate) v += ld1(o);
                st1(o, v);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(S::kColumns));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(S::kColumns));
    }
}

// ------------------------------------------------------------------------------------------
// few rows of a (tokens): no tensor cores
//
// A kernel of tensor-core tiles takes longer to set up and join than to read a small b (4096 x 1024: 3.4
// us, here one row 2.5, four 3.0; 6400 x 1600: 4.1, here one row 3.8, two 4.1, four 4.7; 8192 x 8192: 8.0,
// here 10.7, which instructions bound: 2 a weight to make bytes of codes). Twice a code's value is a whole
// number of at most 12: a block's 32 products are exact in integers (dp4a), and only their sum is
// scaled, in fp32. x: a in 4 bits, or plain, quantised here as onebit_mx4_quantize does (to nearest).
//
// A thread block takes 32 rows of b, warp w rows w, w + 32, w + 64 and w + 96 of eight, whose exponents
// lie in the same 16 bytes; a lane takes every 32nd block of them. a is held in shared memory as bytes,
// kFewCols columns at a time.

constexpr int kFewRows = 4;               // of a, at most
constexpr int kFewCols = 8192;
constexpr int kFewBlocks = kFewCols / kMxBlk;

struct Mx4FewArgs {
    const void* x;             // codes, or values with rows ld apart
    const uint8_t* xs;
    int64_t ldx;
    const uint8_t *b, *sb;
    void* out;
    int64_t ld;
    int32_t m, n, k;
    int32_t accumulate, vec;   // vec: blocks of x's rows are aligned to 32 bytes
};

// Eight codes as 16 more than twice their values. No byte has its top bit set: a byte permutation with
// a code as its selector takes the byte of its magnitude, or 0 if the sign is set (it then repeats the
// top bit), and with the sign turned over the other way round.
__device__ __forceinline__ void biased8(uint32_t c, uint32_t& lo, uint32_t& hi) {
    const uint32_t t = c ^ 0x88888888u;
    lo = prmt(0x13121110u, 0x1c181614u, c) | prmt(0x0d0e0f10u, 0x04080a0cu, t);
    hi = prmt(0x13121110u, 0x1c181614u, c >> 16) | prmt(0x0d0e0f10u, 0x04080a0cu, t >> 16);
}
// ... without what is added (bytes of 4 to 28 less 16: nothing is borrowed but within a byte's top bit).
__device__ __forceinline__ uint32_t unbiased4(uint32_t v) {
    return ((v | 0x80808080u) - 0x10101010u) ^ 0x80808080u;
}

template <int MT, typename XT, typename OT>
__global__ void __launch_bounds__(kMxThreads, 2) k_mx4_few(const Mx4FewArgs p) {
    constexpr bool kPlain = sizeof(XT) > 1;
    after_what_is_ahead();
    // a block's two halves change places in every other four blocks: eight lanes read different banks
    __shared__ uint4 xv[MT][2 * kFewBlocks];
    __shared__ float xf[MT][kFewBlocks];                // an eighth of the block's power of two
    __shared__ int xs[MT][kFewBlocks];                  // what the bias of b's bytes adds, negative
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (p.k + kMxBlk - 1) / kMxBlk;
    const int64_t atoms = mx4_atoms(p.k), pitch = mx4_pitch(p.k);
    const int64_t tile = blockIdx.x >> 2;
    const int r = (blockIdx.x & 3) * 8 + warp;          // within the atom's 32 rows of 16 bytes
    const int64_t n0 = tile * kAtomRows + r;
    const auto stage = [&](int from, int here) {
        for (int i = tid; i < MT * here; i += kMxThreads) {
            const int t = i / here, l = i - t * here, b = from + l;
            uint4 w = make_uint4(0, 0, 0, 0);
            uint32_t k = 0;
            if (t < p.m) {
                if constexpr (kPlain) {
                    const XT* x = static_cast<const XT*>(p.x) + t * p.ldx + (int64_t)b * kMxBlk;
                    const int left = min(p.k - b * kMxBlk, kMxBlk);
                    Values<XT> v;
                    if (p.vec && left == kMxBlk)
                        v.load(x);
                    else
                        v.load_some(x, left);
                    w = encode_block<false>(v, 0u, 0, k);
                } else {
                    w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + t * pitch +
                                                        b * 16);
                    k = p.xs[(b >> 2) * kAtomBytes + atom_at(t, b & 3)];
                }
            }
            const int swap = (l >> 2) & 1;
            const uint32_t c[4] = {w.x, w.y, w.z, w.w};
            uint32_t v[8];
            int sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) biased8(c[j], v[2 * j], v[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = unbiased4(v[j]);
                sum = __dp4a((int)v[j], (int)0xf0f0f0f0, sum);
            }
            xv[t][2 * l + swap] = make_uint4(v[0], v[1], v[2], v[3]);
            xv[t][2 * l + (swap ^ 1)] = make_uint4(v[4], v[5], v[6], v[7]);
            xs[t][l] = sum;
            xf[t][l] = 0.125f * mx4_scale(k);
        }
    };
    // This lane's block b of rows r, r + 32, r + 64, r + 96 of the atom.
    uint4 c[4], e;
    const auto fetch = [&](int b) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            c[g] = make_uint4(0, 0, 0, 0);
            if (n0 + 32 * g < p.n)
                c[g] = *reinterpret_cast<const uint4*>(p.b + (n0 + 32 * g) * pitch + b * 16);
        }
        e = *reinterpret_cast<const uint4*>(p.sb + (tile * atoms + (b >> 2)) * kAtomBytes + r * 16);
    };

    float acc[4][MT];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[g][t] = 0.0f;
    for (int from = 0; from < blocks; from += kFewBlocks) {
        const int here = min(kFewBlocks, blocks - from);
        if (lane < here) fetch(from + lane);
        if (from > 0) __syncthreads();
        stage(from, here);
        __syncthreads();
#pragma unroll 1
        for (int l = lane; l < here; l += 32) {
            const int swap = (l >> 2) & 1;
            uint32_t v[4][8];
            float scales[4];
            {
                const uint32_t ew[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    biased8(c[g].x, v[g][0], v[g][1]);
                    biased8(c[g].y, v[g][2], v[g][3]);
                    biased8(c[g].z, v[g][4], v[g][5]);
                    biased8(c[g].w, v[g][6], v[g][7]);
                    scales[g] = mx4_scale(ew[g] >> (8 * (l & 3)) & 0xffu);
                }
            }
            if (l + 32 < here) fetch(from + l + 32);    // in flight meanwhile
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint4 lo = xv[t][2 * l + swap], hi = xv[t][2 * l + (swap ^ 1)];
                const uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                const float f = xf[t][l];
                const int bias = xs[t][l];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    int s = bias;
#pragma unroll
                    for (int i = 0; i < 8; ++i) s = __dp4a((int)x[i], (int)v[g][i], s);
                    // twice the sum (at most 4608) as a float, by way of 1.5 * 2^24. A scale that
                    // overflows must not make NaN of a sum of 0, a NaN one must; with the largest
                    // number in its place 2 and more still overflow (1 would not).
                    const float twice = __fsub_rn(__int_as_float(s + 0x4bc00000), 25165824.0f);
                    float scale = __fmul_rn(f, scales[g]);
                    asm("min.NaN.f32 %0, %1, %2;" : "=f"(scale) : "f"(scale), "f"(3.402823466e38f));
                    acc[g][t] = __fmaf_rn(twice, scale, acc[g][t]);
                }
            }
        }
    }
    // The lanes' sums, halving the values that a lane holds while there is more than one.
    float s[4 * MT];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int t = 0; t < MT; ++t) s[g * MT + t] = acc[g][t];
    int held = 0, o = 16;
#pragma unroll
    for (int h = 4 * MT; h > 1; h /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < h / 2; ++i) {
            const float keep = up ? s[i + h / 2] : s[i], send = up ? s[i] : s[i + h / 2];
            s[i] = keep + __shfl_xor_sync(kFull, send, o);
        }
        held = 2 * held + (up ? 1 : 0);
    }
#pragma unroll
    for (; o > 0; o /= 2) s[0] += __shfl_xor_sync(kFull, s[0], o);
    const int t = held % MT;
    const int64_t n = n0 + 32 * (held / MT);
    if ((lane & (32 / (4 * MT) - 1)) == 0 && t < p.m && n < p.n) {
        OT* out = static_cast<OT*>(p.out) + t * p.ld + n;
        if (sizeof(OT) == 4 && p.accumulate) s[0] += ld1(out);
        st1(out, s[0]);
    }
}

}  // namespace onebit
