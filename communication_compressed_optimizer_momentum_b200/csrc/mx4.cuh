// mx4.cuh -- host side of the entry points for matrices in microscaled 4-bit floating point
// (onebit_mx4_*): argument checks, the choice of tiles and the launches. Included by onebit_adam.cu.
#pragma once

#include <atomic>

#include "host.h"
#include "kernels_mx4.cuh"
#include "kernels_mx4_matmul.cuh"

namespace {

// The key of the random bits.
uint32_t mx4_key(uint64_t seed) {
    const auto mix = [](uint32_t x) {
        x ^= x >> 16;
        x *= 0x9016D2F5u;
        x ^= x >> 15;
        x *= 0x314549A1u;
        return x ^ (x >> 16);
    };
    return mix(mix((uint32_t)seed + kGolden) ^ (uint32_t)(seed >> 32));
}

constexpr int64_t kMxMost = (int64_t)1 << 30;  // rows or columns

int64_t mx4_code_bytes(int64_t rows, int64_t cols) { return rows * mx4_pitch(cols); }
int64_t mx4_scale_bytes(int64_t rows, int64_t cols) {
    return mx4_atoms(rows) * mx4_atoms(cols) * kAtomBytes;
}

int mx4_shape(const char* where, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > kMxMost || cols > kMxMost) return bad(where, "bad size of a matrix");
    return ONEBIT_OK;
}

// Codes and exponents of one matrix. Empty matrices have neither.
int mx4_matrix(const char* where, int64_t rows, int64_t cols, const void* codes,
               const void* scales) {
    if (rows == 0 || cols == 0) return ONEBIT_OK;
    if (codes == nullptr || scales == nullptr) return bad(where, "null codes or exponents");
    if (!aligned16(codes) || !aligned16(scales))
        return bad(where, "codes or exponents not 16-byte aligned", ONEBIT_ERR_ALIGN);
    return ONEBIT_OK;
}

// A plain matrix with rows `ld` elements apart.
int mx4_plain(const char* where, const char* what, int64_t rows, int64_t cols, const void* x,
              int64_t ld, int64_t w) {
    if (rows == 0 || cols == 0) return ONEBIT_OK;
    if (x == nullptr) return bad(where, std::string("null ") + what);
    if (!aligned_to(x, w))
        return bad(where, std::string(what) + " not aligned to its elements", ONEBIT_ERR_ALIGN);
    // (a matrix whose places pass 2^60 has no memory, and 64 bits would not count its bytes)
    if (rows > 1 && (ld < cols || ld > ((int64_t)1 << 40) || ld > ((int64_t)1 << 60) / rows))
        return bad(where, std::string("bad row stride of ") + what);
    return ONEBIT_OK;
}

int64_t mx4_span(int64_t rows, int64_t cols, int64_t ld, int64_t w) {
    return rows == 0 || cols == 0 ? 0 : ((rows - 1) * ld + cols) * w;
}

// The address ranges of one call, few enough to be compared in pairs (Ranges, for lists, allocates):
// what is written must not overlap anything else.
struct Spans {
    static constexpr int kMost = 8;
    uintptr_t lo[kMost], hi[kMost];
    bool write[kMost];
    int n = 0;
    void add(const void* p, int64_t bytes, bool w) {
        if (p == nullptr || bytes <= 0) return;
        lo[n] = reinterpret_cast<uintptr_t>(p);
        hi[n] = lo[n] + (uintptr_t)bytes;
        write[n++] = w;
    }
    bool clash() const {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((write[i] || write[j]) && lo[i] < hi[j] && lo[j] < hi[i]) return true;
        return false;
    }
};

// Shared memory beyond 48 KB is asked for once for each kernel and device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// How thread blocks of `threads` share rows of `wide` blocks: several rows each, or parts of one.
template <typename A>
int64_t mx4_share(A& a, int64_t rows, int64_t wide, int threads) {
    if (wide <= threads) {
        a.segments = 1;
        a.segment = 0;
        a.rows_per = (int32_t)(threads / wide);
        a.magic = wide > 1 ? (uint32_t)(((uint64_t)1 << 32) / (uint64_t)wide + 1) : 0;
        return ceil_div(rows, a.rows_per);
    }
    a.segments = (int32_t)ceil_div(wide, threads);
    a.segment = (int32_t)ceil_div(wide, a.segments);
    a.rows_per = 0;
    a.magic = 0;
    return rows * a.segments;
}

// A launch that may start before the kernel ahead of it has ended (see after_what_is_ahead).
template <typename... P, typename... A>
int launch_mx4(void (*kernel)(P...), int64_t grid, int threads, int smem, int cluster,
               cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    ONEBIT_CUDA(cudaLaunchKernelEx(&cfg, kernel, args...));
    return ONEBIT_OK;
}

template <typename T, bool SR, bool RES>
int launch_mx4_rows(Mx4QuantArgs a, cudaStream_t st) {
    const int64_t rows = mx4_atoms(a.rows) * kAtomRows, wide = a.col_tiles * 4;
    if constexpr (sizeof(T) == 2 && !RES) {
        const int64_t blocks = mx4_share(a, rows, wide, kMxThreads);
        return launch_mx4(k_mx4_rows<SR>, blocks, kMxThreads, 0, 1, st, a);
    } else {
        const int64_t blocks = mx4_share(a, rows, wide, kMxThreads / 4 * kMxUnits);
        return launch_mx4(k_mx4_rows8<T, SR, RES>, blocks, kMxThreads, 0, 1, st, a);
    }
}

template <typename T, int FORMS, bool SR, bool VEC, bool RES>
int launch_mx4_tile(const Mx4QuantArgs& a, cudaStream_t st) {
    using S = MxTile<typename std::conditional<RES, float, T>::type>;
    static std::atomic<uint64_t> done{0};
    const auto kernel = k_mx4_tile<T, FORMS, SR, VEC, RES>;
    ONEBIT_CUDA(allow_smem(kernel, S::kSmem, done));
    return launch_mx4(kernel, a.col_tiles * S::kParts * mx4_atoms(a.rows), kMxThreads, S::kSmem, 1, st, a);
}

// vec: blocks of x's rows (and of the residual's) are aligned to 32 bytes.
template <typename T, bool SR>
int queue_mx4_quantize(const Mx4QuantArgs& a, bool vec, cudaStream_t st) {
    constexpr int kBoth = kMxRows | kMxColumns;
    if (a.c != nullptr && a.ct != nullptr)
        return vec ? launch_mx4_tile<T, kBoth, SR, true, false>(a, st)
                   : launch_mx4_tile<T, kBoth, SR, false, false>(a, st);
    if (a.ct != nullptr)
        return vec ? launch_mx4_tile<T, kMxColumns, SR, true, false>(a, st)
                   : launch_mx4_tile<T, kMxColumns, SR, false, false>(a, st);
    if (a.e != nullptr)
        return vec ? launch_mx4_rows<T, SR, true>(a, st)
                   : launch_mx4_tile<T, kMxRows, SR, false, true>(a, st);
    return vec ? launch_mx4_rows<T, SR, false>(a, st)
               : launch_mx4_tile<T, kMxRows, SR, false, false>(a, st);
}

// cuTensorMapEncodeTiled, asked of the runtime: the library links to no driver library.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encode_tiled(EncodeTiled* f) {
    static std::atomic<void*> found{nullptr};
    void* p = found.load(std::memory_order_acquire);
    if (p == nullptr) {
        cudaDriverEntryPointQueryResult q;
        ONEBIT_CUDA(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                     cudaEnableDefault, &q));
        if (q != cudaDriverEntryPointSuccess || p == nullptr)
            return cuda_fail(cudaErrorSymbolNotFound);
        found.store(p, std::memory_order_release);
    }
    *f = reinterpret_cast<EncodeTiled>(p);
    return ONEBIT_OK;
}

// A matrix of rows of `width` elements, `ld` apart, taken in boxes; zeros behind the edges.
int box_map(EncodeTiled encode, CUtensorMap* map, CUtensorMapDataType type, int64_t bytes,
            const void* base, int64_t width, int64_t rows, int64_t ld, int across, int down,
            CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ld * bytes)};
    const cuuint32_t box[2] = {(cuuint32_t)across, (cuuint32_t)down}, ones[2] = {1, 1};
    const CUresult r = encode(map, type, 2, const_cast<void*>(base), dims, strides, box, ones,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ONEBIT_OK : cuda_fail(cudaErrorInvalidValue);
}

// The codes as rows of bytes, in boxes of 128 bytes by `box` rows, and the exponents as a row of words
// for each 128 rows, in boxes of two atoms by `atoms` rows. (Exponents as plain bulk copies of 1 KB, of
// which a stage takes three, hold up the loads.)
int operand_maps(EncodeTiled encode, CUtensorMap* codes_map, CUtensorMap* scales_map,
                 const void* codes, const void* scales, int64_t rows, int64_t cols, int box,
                 int atoms) {
    const int rc = box_map(encode, codes_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, mx4_pitch(cols),
                           rows, mx4_pitch(cols), 128, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc != ONEBIT_OK) return rc;
    return box_map(encode, scales_map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, scales,
                   mx4_atoms(cols) * (kAtomBytes / 4), mx4_atoms(rows),
                   mx4_atoms(cols) * (kAtomBytes / 4), 2 * kAtomBytes / 4, atoms,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
}

struct MmOperands {
    const void *a, *sa, *b, *sb;
    int64_t m, n, k;
    Mx4MatmulArgs args;
};

template <int TM, bool PAIR, typename OT, bool SPLIT>
int launch_mx4_matmul(MmOperands o, int split, cudaStream_t st) {
    using S = MmTile<TM, PAIR, SPLIT>;
    static std::atomic<uint64_t> done{0};
    const auto kernel = k_mx4_matmul<TM, PAIR, OT, SPLIT>;
    ONEBIT_CUDA(allow_smem(kernel, S::kSmem, done));
    EncodeTiled encode;
    int rc = encode_tiled(&encode);
    if (rc != ONEBIT_OK) return rc;
    Mx4Maps maps;
    rc = operand_maps(encode, &maps.a, &maps.sa, o.a, o.sa, o.m, o.k, S::kARows, S::kHalves);
    if (rc == ONEBIT_OK)
        rc = operand_maps(encode, &maps.b, &maps.sb, o.b, o.sb, o.n, o.k, kMmLanes, 1);
    if (rc == ONEBIT_OK && o.args.tma) {
        constexpr bool wide = sizeof(OT) == 4;
        rc = box_map(encode, &maps.out, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     sizeof(OT), o.args.out, o.n, o.m, o.m > 1 ? o.args.ld : round_up(o.n, 8), 32,
                     wide ? kOutRows32 : S::kChunk,
                     wide ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B);
    }
    if (rc != ONEBIT_OK) return rc;
    o.args.tiles_m = (int32_t)ceil_div(o.m, TM);
    o.args.tiles_n = (int32_t)ceil_div(o.n, kMmLanes * S::kGroup);
    const int64_t tiles = (int64_t)o.args.tiles_m * o.args.tiles_n;
    const int64_t grid =
        SPLIT ? tiles * split : std::min<int64_t>(tiles, kSms / S::kGroup) * S::kGroup;
    return launch_mx4(kernel, grid, kMmThreads, S::kSmem, PAIR ? 2 : split, st, maps, o.args);
}

// The tiles of a product: rows of out, and the blocks that share one tile's common axis (1: none do).
struct MmChoice {
    int rows, split;
};
MmChoice choose_tiles(int64_t m, int64_t n, int64_t stages, bool wide) {
    const int64_t tn = ceil_div(n, kMmLanes);
    // Few rows: narrow tiles; what they leave idle takes parts of the common axis, of four stages and
    // more (16 x 4096 from 4096: 6.7 us in four parts, 7.2 in one; from 1024: 7.1 and 4.5).
    const auto narrow = [&](int tm) {
        const int64_t split =
            std::min<int64_t>(std::min<int64_t>(8, kSms / (tn * ceil_div(m, tm))), stages / 4);
        return MmChoice{tm, (int)std::max<int64_t>(split, 1)};
    };
    if (m <= 16) return narrow(16);
    // What a launch takes, in 10 ns, as measured: once, and a round of tiles by its stages and by what
    // it writes. (4096 x 4096 from 1024: tiles of 64 rows 14.0 us, 128 10.2, 256 10.1; 1024 x 1024 from
    // 1024: 5.0, 5.5, 7.3; 512 x 4096 from 4096: 13.4, 8.9, 11.2.)
    const auto cost = [&](int tm, int group, int64_t once, int64_t stage, int64_t tile) {
        const int64_t tiles = ceil_div(m, tm) * ceil_div(n, kMmLanes * group);
        return once + ceil_div(tiles, kSms / group) * (stages * stage + tile);
    };
    const int64_t c32 = cost(32, 1, 390, 20, 30), c64 = cost(64, 1, 390, 22, wide ? 60 : 40),
                  c128 = cost(128, 1, 400, 24, wide ? 120 : 60),
                  c256 = cost(256, 2, 590, 31, wide ? 250 : 80);
    const int64_t best = std::min(std::min(c32, c64), std::min(c128, c256));
    if (best == c256) return {256, 1};
    if (best == c128) return {128, 1};
    if (best == c64) return {64, 1};
    return narrow(32);
}

template <typename OT>
int queue_mx4_matmul(const MmOperands& o, cudaStream_t st) {
    const MmChoice t = choose_tiles(o.m, o.n, o.args.stages, sizeof(OT) == 4);
    if (t.rows == 256) return launch_mx4_matmul<256, true, OT, false>(o, 1, st);
    if (t.rows == 128) return launch_mx4_matmul<128, false, OT, false>(o, 1, st);
    if (t.rows == 64) return launch_mx4_matmul<64, false, OT, false>(o, 1, st);
    if (t.rows == 32)
        return t.split > 1 ? launch_mx4_matmul<32, false, OT, true>(o, t.split, st)
                           : launch_mx4_matmul<32, false, OT, false>(o, 1, st);
    return t.split > 1 ? launch_mx4_matmul<16, false, OT, true>(o, t.split, st)
                       : launch_mx4_matmul<16, false, OT, false>(o, 1, st);
}

// The limit of a product's waits (onebit_internal_mx4_wait).
std::atomic<uint64_t> g_mx4_wait_ns{kMmWaitNs};

// At most kFewRows rows of x, which is in 4 bits (XT uint8_t) or plain.
template <typename XT, typename OT>
int queue_mx4_few(const Mx4FewArgs& a, cudaStream_t st) {
    const auto kernel = a.m == 1   ? k_mx4_few<1, XT, OT>
                        : a.m == 2 ? k_mx4_few<2, XT, OT>
                                   : k_mx4_few<4, XT, OT>;
    return launch_mx4(kernel, 4 * mx4_atoms(a.n), kMxThreads, 0, 1, st, a);
}
template <typename XT>
int queue_mx4_few(const Mx4FewArgs& a, int32_t dtype, cudaStream_t st) {
    return dtype == ONEBIT_F32 ? queue_mx4_few<XT, float>(a, st)
                               : queue_mx4_few<XT, __nv_bfloat16>(a, st);
}

// out, m x n with rows ld apart, of no common axis: zeros.
int mx4_clear(void* out, int64_t m, int64_t n, int64_t ld, int64_t w, cudaStream_t st) {
    ONEBIT_CUDA(cudaMemset2DAsync(out, (size_t)((m > 1 ? ld : n) * w), 0, (size_t)(n * w), (size_t)m, st));
    return ONEBIT_OK;
}

// Whether few rows are multiplied without the tensor cores: up to 6M weights, between those where one to
// four rows gain (4M) and those where four rows lose (10M, 4.7 us against 4.1, and one gains 0.3; see
// k_mx4_few), and up to 12M where that saves a launch that quantises them (6400 x 1600: one row 4.1 us
// against 5.4 in two launches, four 5.4 against 5.6).
bool mx4_few(int64_t m, int64_t n, int64_t k, bool plain) {
    return m <= kFewRows && n * k <= (plain ? (int64_t)3 << 22 : (int64_t)3 << 21);
}

// The product, once everything is checked (k > 0).
int mx4_product(int64_t m, int64_t n, int64_t k, const void* a, const void* sa, const void* b,
                const void* sb, void* out, int32_t dtype, int64_t ld, int32_t accumulate, bool few,
                cudaStream_t st) {
    if (few) {
        Mx4FewArgs f{};
        f.x = a;
        f.xs = static_cast<const uint8_t*>(sa);
        f.b = static_cast<const uint8_t*>(b);
        f.sb = static_cast<const uint8_t*>(sb);
        f.out = out;
        f.ld = ld;
        f.m = (int32_t)m;
        f.n = (int32_t)n;
        f.k = (int32_t)k;
        f.accumulate = accumulate;
        return queue_mx4_few<uint8_t>(f, dtype, st);
    }
    MmOperands o{a, sa, b, sb, m, n, k, {}};
    o.args.out = out;
    o.args.ld = ld;
    o.args.m = (int32_t)m;
    o.args.n = (int32_t)n;
    o.args.steps = (int32_t)ceil_div(k, 64);
    o.args.stages = (int32_t)ceil_div(k, kStageCols);
    o.args.accumulate = accumulate;
    o.args.wait_ns = g_mx4_wait_ns.load(std::memory_order_relaxed);
    o.args.tma = aligned16(out) && (m == 1 || (ld * width(dtype) % 16 == 0 &&
                                               ld * width(dtype) < (int64_t)1 << 40));
    return dtype == ONEBIT_F32 ? queue_mx4_matmul<float>(o, st)
                               : queue_mx4_matmul<__nv_bfloat16>(o, st);
}

// Tiles are counted in 32 bits.
int mx4_tiles(const char* where, int64_t rows, int64_t cols) {
    return mx4_atoms(rows) * mx4_atoms(cols) > ((int64_t)1 << 29) ? bad(where, "bad size of a matrix")
                                                                  : ONEBIT_OK;
}
int mx4_out_size(const char* where, int64_t m, int64_t n) {
    return ceil_div(m, 16) * ceil_div(n, kMmLanes) > ((int64_t)1 << 30) ? bad(where, "out is too large")
                                                                      : ONEBIT_OK;
}

int mx4_quantize(int64_t rows, int64_t cols, const void* x, int32_t dtype,
                 int64_t ld, uint8_t* codes, uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                 int32_t stochastic, uint64_t seed, float* residual, int64_t ld_residual,
                 cudaStream_t st) {
    Mx4QuantArgs a{};
    a.x = x;
    a.ld = ld;
    a.rows = rows;
    a.cols = cols;
    a.e = residual;
    a.lde = ld_residual;
    a.c = codes;
    a.s = scales;
    a.ct = codes_t;
    a.st = scales_t;
    a.key = mx4_key(seed);
    a.tkey = mx4_key(seed + 1);
    a.col_tiles = mx4_atoms(cols);
    const int64_t w = width(dtype);
    const bool vec = aligned_to(x, 32) && (rows == 1 || ld * w % 32 == 0) && aligned_to(residual, 32) &&
                     (residual == nullptr || rows == 1 || ld_residual % 8 == 0);
    if (dtype == ONEBIT_F32)
        return stochastic ? queue_mx4_quantize<float, true>(a, vec, st)
                          : queue_mx4_quantize<float, false>(a, vec, st);
    return stochastic ? queue_mx4_quantize<__nv_bfloat16, true>(a, vec, st)
                      : queue_mx4_quantize<__nv_bfloat16, false>(a, vec, st);
}

}  // namespace

extern "C" {

int onebit_mx4_layout(int64_t rows, int64_t cols, int64_t* code_bytes, int64_t* scale_bytes) {
    return guarded([&]() -> int {
        const char* where = "onebit_mx4_layout";
        const int rc = mx4_shape(where, rows, cols);
        if (rc != ONEBIT_OK) return rc;
        if (code_bytes == nullptr || scale_bytes == nullptr) return bad(where, "null result");
        *code_bytes = mx4_code_bytes(rows, cols);
        *scale_bytes = mx4_scale_bytes(rows, cols);
        return ONEBIT_OK;
    });
}

int onebit_mx4_quantize(int64_t rows, int64_t cols, const void* x, int32_t dtype, int64_t ld,
                        uint8_t* codes, uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                        int32_t stochastic, uint64_t seed, float* residual, int64_t ld_residual,
                        void* stream) {
    return guarded([&]() -> int {
        const char* where = "onebit_mx4_quantize";
        int rc = mx4_shape(where, rows, cols);
        if (rc != ONEBIT_OK) return rc;
        if (!known_dtype(dtype)) return bad(where, "unknown type");
        if (stochastic != 0 && stochastic != 1) return bad(where, "stochastic must be 0 or 1");
        if (rows == 0 || cols == 0) return ONEBIT_OK;
        if (codes == nullptr && codes_t == nullptr) return bad(where, "neither codes nor codes_t");
        if (residual != nullptr && (codes == nullptr || codes_t != nullptr))
            return bad(where, "a residual goes with codes alone");
        rc = mx4_tiles(where, rows, cols);
        if (rc == ONEBIT_OK) rc = mx4_plain(where, "x", rows, cols, x, ld, width(dtype));
        if (rc == ONEBIT_OK && codes != nullptr) rc = mx4_matrix(where, rows, cols, codes, scales);
        if (rc == ONEBIT_OK && codes_t != nullptr)
            rc = mx4_matrix(where, cols, rows, codes_t, scales_t);
        if (rc == ONEBIT_OK && residual != nullptr)
            rc = mx4_plain(where, "residual", rows, cols, residual, ld_residual, 4);
        if (rc != ONEBIT_OK) return rc;
        Spans spans;
        spans.add(x, mx4_span(rows, cols, ld, width(dtype)), false);
        if (codes != nullptr) {
            spans.add(codes, mx4_code_bytes(rows, cols), true);
            spans.add(scales, mx4_scale_bytes(rows, cols), true);
        }
        if (codes_t != nullptr) {
            spans.add(codes_t, mx4_code_bytes(cols, rows), true);
            spans.add(scales_t, mx4_scale_bytes(cols, rows), true);
        }
        if (residual != nullptr) spans.add(residual, mx4_span(rows, cols, ld_residual, 4), true);
        if (spans.clash()) return bad(where, "what is written overlaps something else");
        return mx4_quantize(rows, cols, x, dtype, ld, codes, scales, codes_t, scales_t,
                            stochastic, seed, residual, ld_residual, as_stream(stream));
    });
}

int onebit_mx4_dequantize(int64_t rows, int64_t cols, const uint8_t* codes, const uint8_t* scales,
                          void* out, int32_t dtype, int64_t ld, void* stream) {
    return guarded([&]() -> int {
        const char* where = "onebit_mx4_dequantize";
        int rc = mx4_shape(where, rows, cols);
        if (rc != ONEBIT_OK) return rc;
        if (!known_dtype(dtype)) return bad(where, "unknown type");
        rc = mx4_matrix(where, rows, cols, codes, scales);
        if (rc == ONEBIT_OK) rc = mx4_plain(where, "out", rows, cols, out, ld, width(dtype));
        if (rc != ONEBIT_OK || rows == 0 || cols == 0) return rc;
        rc = mx4_tiles(where, rows, cols);
        if (rc != ONEBIT_OK) return rc;
        Spans spans;
        spans.add(codes, mx4_code_bytes(rows, cols), false);
        spans.add(scales, mx4_scale_bytes(rows, cols), false);
        spans.add(out, mx4_span(rows, cols, ld, width(dtype)), true);
        if (spans.clash()) return bad(where, "out overlaps the codes or exponents");
        Mx4DequantArgs a{};
        a.c = codes;
        a.s = scales;
        a.out = out;
        a.ld = ld;
        a.rows = rows;
        a.cols = cols;
        a.col_tiles = mx4_atoms(cols);
        const int64_t w = width(dtype);
        const bool vec = aligned_to(out, 32) && (rows == 1 || ld * w % 32 == 0);
        const bool wide = dtype == ONEBIT_F32;
        const int64_t grid = mx4_share(
            a, rows, mx4_blocks(cols), wide && vec ? kMxThreads / 4 * kMxUnits : kMxThreads);
        const cudaStream_t st = as_stream(stream);
        const auto kernel = wide ? (vec ? k_mx4_dequantize8 : k_mx4_dequantize<float, false>)
                            : vec ? k_mx4_dequantize<__nv_bfloat16, true>
                                  : k_mx4_dequantize<__nv_bfloat16, false>;
        return launch_mx4(kernel, grid, kMxThreads, 0, 1, st, a);
    });
}

int onebit_mx4_matmul(int64_t m, int64_t n, int64_t k, const uint8_t* a_codes,
                      const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales,
                      void* out, int32_t dtype, int64_t ld, int32_t accumulate, void* stream) {
    return guarded([&]() -> int {
        const char* where = "onebit_mx4_matmul";
        int rc = mx4_shape(where, m, k);
        if (rc == ONEBIT_OK) rc = mx4_shape(where, n, k);
        if (rc != ONEBIT_OK) return rc;
        if (!known_dtype(dtype)) return bad(where, "unknown type");
        if (accumulate != 0 && accumulate != 1) return bad(where, "accumulate must be 0 or 1");
        if (accumulate && dtype != ONEBIT_F32) return bad(where, "accumulation needs a float32 out");
        if (m == 0 || n == 0) return ONEBIT_OK;
        rc = mx4_matrix(where, m, k, a_codes, a_scales);
        if (rc == ONEBIT_OK) rc = mx4_matrix(where, n, k, b_codes, b_scales);
        if (rc == ONEBIT_OK) rc = mx4_plain(where, "out", m, n, out, ld, width(dtype));
        if (rc == ONEBIT_OK) rc = mx4_out_size(where, m, n);
        if (rc != ONEBIT_OK) return rc;
        Spans spans;
        if (k > 0) {
            spans.add(a_codes, mx4_code_bytes(m, k), false);
            spans.add(a_scales, mx4_scale_bytes(m, k), false);
            spans.add(b_codes, mx4_code_bytes(n, k), false);
            spans.add(b_scales, mx4_scale_bytes(n, k), false);
        }
        spans.add(out, mx4_span(m, n, ld, width(dtype)), true);
        if (spans.clash()) return bad(where, "out overlaps an operand");
        const cudaStream_t st = as_stream(stream);
        if (k == 0) return accumulate ? ONEBIT_OK : mx4_clear(out, m, n, ld, width(dtype), st);
        return mx4_product(m, n, k, a_codes, a_scales, b_codes, b_scales, out, dtype, ld, accumulate,
                           mx4_few(m, n, k, false), st);
    });
}

int onebit_mx4_linear(int64_t m, int64_t n, int64_t k, const void* x, int32_t x_dtype, int64_t ld_x,
                      const uint8_t* b_codes, const uint8_t* b_scales, uint8_t* a_codes,
                      uint8_t* a_scales, uint8_t* a_codes_t, uint8_t* a_scales_t, void* out,
                      int32_t dtype, int64_t ld, void* stream) {
    return guarded([&]() -> int {
        const char* where = "onebit_mx4_linear";
        int rc = mx4_shape(where, m, k);
        if (rc == ONEBIT_OK) rc = mx4_shape(where, n, k);
        if (rc != ONEBIT_OK) return rc;
        if (!known_dtype(x_dtype) || !known_dtype(dtype)) return bad(where, "unknown type");
        const bool kept = a_codes_t != nullptr && m > 0 && k > 0;
        const bool few = !kept && mx4_few(m, n, k, true);
        rc = mx4_plain(where, "x", m, k, x, ld_x, width(x_dtype));
        if (rc == ONEBIT_OK && !few) rc = mx4_matrix(where, m, k, a_codes, a_scales);
        if (rc == ONEBIT_OK && kept) rc = mx4_matrix(where, k, m, a_codes_t, a_scales_t);
        if (rc == ONEBIT_OK && m > 0) rc = mx4_matrix(where, n, k, b_codes, b_scales);
        if (rc == ONEBIT_OK) rc = mx4_plain(where, "out", m, n, out, ld, width(dtype));
        if (rc == ONEBIT_OK) rc = mx4_out_size(where, m, n);
        if (rc == ONEBIT_OK) rc = mx4_tiles(where, m, k);
        if (rc != ONEBIT_OK || m == 0) return rc;
        Spans spans;
        if (k > 0) {
            spans.add(x, mx4_span(m, k, ld_x, width(x_dtype)), false);
            if (n > 0) {
                spans.add(b_codes, mx4_code_bytes(n, k), false);
                spans.add(b_scales, mx4_scale_bytes(n, k), false);
            }
            if (!few) {
                spans.add(a_codes, mx4_code_bytes(m, k), true);
                spans.add(a_scales, mx4_scale_bytes(m, k), true);
            }
            if (kept) {
                spans.add(a_codes_t, mx4_code_bytes(k, m), true);
                spans.add(a_scales_t, mx4_scale_bytes(k, m), true);
            }
        }
        spans.add(out, mx4_span(m, n, ld, width(dtype)), true);
        if (spans.clash()) return bad(where, "what is written overlaps something else");
        const cudaStream_t st = as_stream(stream);
        if (k == 0) return n > 0 ? mx4_clear(out, m, n, ld, width(dtype), st) : ONEBIT_OK;
        if (few) {
            if (n == 0) return ONEBIT_OK;
            Mx4FewArgs f{};
            f.x = x;
            f.ldx = ld_x;
            f.b = b_codes;
            f.sb = b_scales;
            f.out = out;
            f.ld = ld;
            f.m = (int32_t)m;
            f.n = (int32_t)n;
            f.k = (int32_t)k;
            f.vec = aligned_to(x, 32) && (m == 1 || ld_x * width(x_dtype) % 32 == 0);
            return x_dtype == ONEBIT_F32 ? queue_mx4_few<float>(f, dtype, st)
                                         : queue_mx4_few<__nv_bfloat16>(f, dtype, st);
        }
        rc = mx4_quantize(m, k, x, x_dtype, ld_x, a_codes, a_scales, a_codes_t, a_scales_t, 0, 0,
                          nullptr, 0, st);
        if (rc != ONEBIT_OK || n == 0) return rc;
        // (with the kernel that takes x as it is, the same sums)
        return mx4_product(m, n, k, a_codes, a_scales, b_codes, b_scales, out, dtype, ld, 0,
                           mx4_few(m, n, k, true), st);
    });
}

int onebit_mx4_linear_needs(int64_t m, int64_t n, int64_t k) { return mx4_few(m, n, k, true) ? 0 : 1; }

// For tests, not part of the C ABI: what a product of these sizes (none 0) is made with. rows: of a tile
// of out, 0 without the tensor cores; split: blocks that share a tile's common axis. Host only.
void onebit_internal_mx4_tiles(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t* rows,
                               int32_t* split) {
    const MmChoice t = mx4_few(m, n, k, false)
                           ? MmChoice{0, 1}
                           : choose_tiles(m, n, ceil_div(k, kStageCols), dtype == ONEBIT_F32);
    *rows = t.rows;
    *split = t.split;
}

// For tests, not part of the C ABI: after how many ns the waits of products that are queued from now on
// give up; 0: the 20 s that they have otherwise. Host only.
void onebit_internal_mx4_wait(uint64_t ns) { g_mx4_wait_ns.store(ns != 0 ? ns : kMmWaitNs); }

int onebit_mx4_status(uint32_t* flags, void* stream) {
    return guarded([&]() -> int {
        if (flags == nullptr) return bad("onebit_mx4_status", "null flags");
        const cudaStream_t st = as_stream(stream);
        ONEBIT_CUDA(cudaMemcpyFromSymbolAsync(flags, g_mx4_status, 4, 0, cudaMemcpyDeviceToHost, st));
        ONEBIT_CUDA(cudaStreamSynchronize(st));
        return ONEBIT_OK;
    });
}

}  // extern "C"
