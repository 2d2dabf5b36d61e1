// kernels_mx4.cuh -- matrices in microscaled 4-bit floating point for B200 (sm_100a): quantising and
// reading back (kernels_mx4_matmul.cuh has the products).
//
// A matrix of rows x cols is held as codes (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6; two a byte, the even column in the lower half, rows of 16 * ceil(cols / 32) bytes) and
// one power of two for each block of 32 consecutive columns of a row (a byte, the exponent plus 127;
// 255: the whole block is NaN). The exponents lie in ATOMS of 128 rows by 4 blocks, 512 bytes: row r
// and block b of an atom at (r % 32) * 16 + (r / 32) * 4 + b. That is the order in which the tensor
// cores take them: one 32 x 128 bit copy from shared memory puts an atom into four columns of tensor
// memory, and the two blocks of one 64-column instruction are the lower or the upper half of a word.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.cuh"
#include "kernels_adamw.cuh"

namespace onebit {

constexpr int kMxBlk = 32;        // columns that share an exponent
constexpr int kAtomRows = 128;    // of an atom of exponents
constexpr int kAtomCols = 128;    // columns: four blocks
constexpr int kAtomBytes = 512;
constexpr int kMxNan = 255;

__host__ __device__ inline int64_t mx4_blocks(int64_t cols) { return (cols + kMxBlk - 1) / kMxBlk; }
__host__ __device__ inline int64_t mx4_pitch(int64_t cols) { return 16 * mx4_blocks(cols); }
__host__ __device__ inline int64_t mx4_atoms(int64_t n) { return (n + kAtomCols - 1) / kAtomCols; }

// These kernels are queued so that they may start before the one ahead of them in the stream has ended:
// each first lets its own follower start likewise, and touches memory only once everything ahead is done
// and visible. What lies between two kernels (launch, barriers, tensor memory) overlaps then.
__device__ __forceinline__ void after_what_is_ahead() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Byte of the exponent of a row and a block within its atom.
__device__ __forceinline__ int atom_at(int r, int b) { return (r & 31) * 16 + (r >> 5) * 4 + b; }

// ------------------------------------------------------------------------------------------
// quantising
//
// A block's exponent is the smallest with which its largest magnitude does not exceed 6:
//   k = max(E - 2, 0), E the biased exponent of the largest magnitude, one more if its mantissa is
//   above 1.5 (the sum with 0x3fffff carries then);  magnitudes above 1.5 * 2^127, infinities and NaN
//   (E = 255) make the block NaN.
// Nothing saturates, so that stochastic rounding has no bias. z = x * 2^(127 - k) is exact (a power
// of two) unless it is below 2^-126, far below the smallest code's half.

__device__ __forceinline__ uint32_t mx4_exponent(uint32_t most) {
    const uint32_t e = (most + 0x3fffffu) >> 23;
    return e >= 255u ? (uint32_t)kMxNan : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - k), 0 for a NaN block (whose codes are then 0).
__device__ __forceinline__ float mx4_inverse(uint32_t k) {
    return k == kMxNan ? 0.0f : __uint_as_float((254u - k) << 23);
}
// 2^(k - 127), NaN for a NaN block.
__device__ __forceinline__ float mx4_scale(uint32_t k) {
    return k == kMxNan ? __uint_as_float(0x7fffffffu)
                       : __uint_as_float(k > 0u ? k << 23 : 0x00400000u);
}

// Eight codes, rounded to nearest (ties to the even code): element i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t encode8_nearest(const float (&z)[8]) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
    return r;
}

// Eight codes, rounded up with the probability of the remainder in 16 bits. y = z * 2^-126 (rounded
// toward zero: a remainder keeps 22 bits) lines the codes up with bits 24 to 22 of an fp32 pattern,
// subnormal ones too; the random bits are added below them. |z| <= 6 cannot carry beyond the largest
// code. w: the random word of the group of eight. Instructions bound it, 15 a value with all that
// belongs to it (8192 x 4096 bf16 in both forms: 34 us, 16 at the rate of HBM).
__device__ __forceinline__ uint32_t encode8_stochastic(const float (&y)[8], uint32_t w) {
    uint32_t r = 0;
#pragma unroll
    for (int p = 3; p >= 0; --p) {
        uint32_t x = w + (uint32_t)(p + 1) * kGolden;
        x ^= x >> 15;
        x *= 0x8A8866C7u;
        const uint32_t u[2] = {x >> 16, (x ^ (x >> 16)) & 0xffffu};
#pragma unroll
        for (int h = 1; h >= 0; --h) {
            const uint32_t t = __float_as_uint(y[2 * p + h]) + u[h] * 64u;
            r = __funnelshift_l((t << 6) | (t & 0x80000000u), r, 4);   // sign and code on top
        }
    }
    return r;
}

// Values to codes in a block of exponent k, eight at a time: GROUPS groups; get(i): the values; word(g):
// the random word of a group.
template <bool SR, int GROUPS, typename F, typename W>
__device__ __forceinline__ void encode_groups(F&& get, W&& word, uint32_t k, uint32_t (&codes)[GROUPS]) {
    const auto all = [&](auto&& scaled) {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            float z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = scaled(get(8 * g + i));
            if constexpr (SR)
                codes[g] = encode8_stochastic(z, word(g));
            else
                codes[g] = encode8_nearest(z);
            if (k == kMxNan) codes[g] = 0u;
        }
    };
    const float inv = mx4_inverse(k);
    if constexpr (!SR) {
        all([&](float v) { return v * inv; });
    } else if (k <= 127u) {            // one factor where fp32 has it, 2^(1 - k)
        const float f = k == 0u ? 2.0f : __uint_as_float((128u - k) << 23);
        all([&](float v) { return __fmul_rz(v, f); });
    } else {
        all([&](float v) { return __fmul_rz(v * inv, 0x1p-126f); });
    }
}

// The larger magnitudes of two pairs of bf16, or NaN; the result's signs mean nothing.
__device__ __forceinline__ uint32_t max_magnitude2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A block of 32 values, as it is loaded.
template <typename T>
struct Values;
template <>
struct Values<float> {
    float v[32];
    __device__ __forceinline__ float get(int i) const { return v[i]; }
    __device__ __forceinline__ uint32_t most() const {
        float m[4] = {fabsf(v[0]), fabsf(v[1]), fabsf(v[2]), fabsf(v[3])};
#pragma unroll
        for (int i = 4; i < 32; ++i) m[i & 3] = max_nan(m[i & 3], fabsf(v[i]));
        return __float_as_uint(max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]))) & 0x7fffffffu;
    }
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float t[8];
            ld8(p + 8 * g, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * g + i] = t[i];
        }
    }
    __device__ __forceinline__ void load_some(const float* p, int n) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
};
template <>
struct Values<__nv_bfloat16> {
    uint32_t w[16];
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ uint32_t most() const {
        uint32_t m[2] = {w[0], w[1]};
#pragma unroll
        for (int i = 2; i < 16; ++i) m[i & 1] = max_magnitude2(m[i & 1], w[i]);
        const uint32_t x = max_magnitude2(m[0], m[1]) & 0x7fff7fffu;
        return max(x << 16, x & 0xffff0000u);
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
            asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(w[8 * g]), "=r"(w[8 * g + 1]), "=r"(w[8 * g + 2]),
                           "=r"(w[8 * g + 3]), "=r"(w[8 * g + 4]), "=r"(w[8 * g + 5]),
                           "=r"(w[8 * g + 6]), "=r"(w[8 * g + 7])
                         : "l"(p + 16 * g));
    }
    __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            w[i] = (2 * i < n ? q[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
    }
};

// Codes of a block of exponent k; get(i): its values; G: its first place / 8; key: of the random bits.
template <bool SR, typename F>
__device__ __forceinline__ uint4 encode32(F&& get, uint32_t k, uint32_t key, int64_t G) {
    const uint32_t kh = SR ? key + (uint32_t)(G >> 32) * kGolden + (uint32_t)G : 0u;
    uint32_t w[4];
    encode_groups<SR>(get, [&](int g) { return mix32(kh + g); }, k, w);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// The same with the exponent that the block takes.
template <bool SR, typename V>
__device__ __forceinline__ uint4 encode_block(const V& v, uint32_t key, int64_t G, uint32_t& k) {
    k = mx4_exponent(v.most());
    return encode32<SR>([&](int i) { return v.get(i); }, k, key, G);
}

// A byte permutation whose selectors are four bits: the upper one repeats the byte's top bit
// (__byte_perm leaves it out).
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// Eight codes (a word) as bf16 values times a power of two: both bytes of a magnitude come from a
// table of eight, the signs go on top. Exact: bf16 holds every such value.
__device__ __forceinline__ uint4 decode8(uint32_t c, uint32_t scale2) {
    uint32_t o[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t x = h == 0 ? c : c >> 16, sel = x & 0x7777u;
        const uint32_t hi = prmt(0x3f3f3f00u, 0x40404040u, sel);
        const uint32_t lo = prmt(0xc0800000u, 0xc0804000u, sel);
        const uint32_t even = __byte_perm(lo, hi, 0x5140) | ((x & 0x8u) << 12) | ((x & 0x80u) << 24);
        const uint32_t odd =
            __byte_perm(lo, hi, 0x7362) | ((x & 0x800u) << 4) | ((x & 0x8000u) << 16);
        const uint32_t two[2] = {even, odd};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[2 * h + i]) : "r"(two[i]), "r"(scale2));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
// 2^(k - 127), NaN for a NaN block, twice in bf16.
__device__ __forceinline__ uint32_t mx4_scale2(uint32_t k) {
    const uint32_t h = k == kMxNan ? 0x7fffu : k > 0u ? k << 7 : 0x0040u;
    return h | h << 16;
}
__device__ __forceinline__ float bf16_at(const uint4& w, int i) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    return __uint_as_float((i & 1) ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
}

struct Mx4QuantArgs {
    const void* x;
    int64_t ld, rows, cols;
    float* e;                  // residual (or null)
    int64_t lde;
    uint8_t *c, *s;            // the matrix: codes and exponents
    uint8_t *ct, *st;          // the transposed matrix
    uint32_t key, tkey;        // of the random bits: the matrix's, the transposed one's
    int64_t col_tiles;         // of 128
    // k_mx4_rows: thread blocks take `rows_per` rows (segments = 1), or `segment` blocks of one row
    int32_t segments, segment, rows_per;
    uint32_t magic;            // 2^32 / (blocks of a row, up to a multiple of four), rounded up
};

constexpr int kMxRows = 1, kMxColumns = 2;   // forms
constexpr int kMxThreads = 256;

// The matrix itself, from rows whose blocks are aligned to 32 bytes. A thread takes UNITS of what is 32
// bytes or more: bf16 a whole block, so that nothing is exchanged (8192 x 8192: 27 us; eight values a
// thread, whose instructions bound it: 48); fp32, or with a residual, eight values, four lanes a block,
// so that a warp's accesses are contiguous (a block a thread, whose accesses touch each line of memory
// four times: 51 us against 45).
struct MxPlace {
    int64_t row;
    int b;
    bool in;
};
// Block `slot` of this thread block.
__device__ __forceinline__ MxPlace mx4_place(int slot, int wide, int32_t segments, int32_t segment,
                                             int32_t rows_per, uint32_t magic, int64_t rows) {
    MxPlace p;
    if (segments == 1) {
        const int r = magic != 0 ? (int)__umulhi((uint32_t)slot, magic) : slot;
        p.b = slot - r * wide;
        p.row = (int64_t)blockIdx.x * rows_per + r;
        p.in = r < rows_per && p.row < rows;
    } else {
        const uint32_t row = blockIdx.x / (uint32_t)segments;
        p.row = row;
        p.b = (int)(blockIdx.x - row * (uint32_t)segments) * segment + slot;
        p.in = slot < segment && p.b < wide;
    }
    return p;
}

template <bool SR>
__global__ void __launch_bounds__(kMxThreads) k_mx4_rows(const Mx4QuantArgs a) {
    after_what_is_ahead();
    const int wide = (int)a.col_tiles * 4;          // blocks of a row, those of no column among them
    const MxPlace t = mx4_place(threadIdx.x, wide, a.segments, a.segment, a.rows_per, a.magic,
                                mx4_atoms(a.rows) * kAtomRows);
    if (!t.in) return;
    const int64_t pitch = mx4_pitch(a.cols), col = (int64_t)t.b * kMxBlk;
    uint32_t k = 0;
    if (t.row < a.rows && col < a.cols) {
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + t.row * a.ld + col;
        const int n = (int)min(a.cols - col, (int64_t)kMxBlk);
        Values<__nv_bfloat16> v;
        if (n == kMxBlk)
            v.load(x);
        else
            v.load_some(x, n);
        *reinterpret_cast<uint4*>(a.c + t.row * pitch + col / 2) =
            encode_block<SR>(v, a.key, (t.row * pitch) / 4 + t.b * 4, k);
    }
    a.s[((t.row >> 7) * a.col_tiles + (t.b >> 2)) * kAtomBytes + atom_at((int)(t.row & 127), t.b & 3)] =
        (uint8_t)k;
}

// Eight values from `col` on, zeros from `cols` on.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t left, float (&o)[8]) {
    if (left >= 8) {
        ld8(p, o);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = i < left ? ld1(p + i) : 0.0f;
    }
}

// Eight values of a block that four lanes share: codes and the block's exponent.
template <bool SR>
__device__ __forceinline__ uint32_t encode_quarter(const float (&v)[8], uint32_t key, int64_t G,
                                                   uint32_t& k) {
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
    uint32_t most = __float_as_uint(m) & 0x7fffffffu;
    most = max(most, __shfl_xor_sync(kFull, most, 1));
    most = max(most, __shfl_xor_sync(kFull, most, 2));
    k = mx4_exponent(most);
    uint32_t w[1];
    encode_groups<SR>([&](int i) { return v[i]; }, [&](int) { return group_word(key, G); }, k, w);
    return w[0];
}

constexpr int kMxUnits = 2;

template <typename T, bool SR, bool RES>
__global__ void __launch_bounds__(kMxThreads) k_mx4_rows8(const Mx4QuantArgs a) {
    after_what_is_ahead();
    const int wide = (int)a.col_tiles * 4, g = threadIdx.x & 3;
    const int64_t pitch = mx4_pitch(a.cols);
    MxPlace t[kMxUnits];
    float v[kMxUnits][8], e[RES ? kMxUnits : 1][8];
#pragma unroll
    for (int u = 0; u < kMxUnits; ++u) {
        t[u] = mx4_place((int)threadIdx.x / 4 + u * (kMxThreads / 4), wide, a.segments, a.segment,
                         a.rows_per, a.magic, mx4_atoms(a.rows) * kAtomRows);
        const int64_t col = (int64_t)t[u].b * kMxBlk + 8 * g;
        const int64_t left = t[u].in && t[u].row < a.rows ? a.cols - col : 0;
        load8(static_cast<const T*>(a.x) + t[u].row * a.ld + col, left, v[u]);
        if constexpr (RES) load8(a.e + t[u].row * a.lde + col, left, e[u]);
    }
#pragma unroll
    for (int u = 0; u < kMxUnits; ++u) {
        const int64_t row = t[u].row;
        const int b = t[u].b;
        const int64_t col = (int64_t)b * kMxBlk + 8 * g;
        const bool in = t[u].in && row < a.rows;
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = __fadd_rn(v[u][i], e[u][i]);
        }
        uint32_t k;
        const uint32_t w = encode_quarter<SR>(v[u], a.key, (row * pitch) / 4 + b * 4 + g, k);
        if (in && col / 2 < pitch) *reinterpret_cast<uint32_t*>(a.c + row * pitch + col / 2) = w;
        if (t[u].in && g == 0)
            a.s[((row >> 7) * a.col_tiles + (b >> 2)) * kAtomBytes + atom_at((int)(row & 127), b & 3)] =
                (uint8_t)k;
        if constexpr (RES) {
            const uint4 q = decode8(w, mx4_scale2(k));
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __fsub_rn(v[u][i], bf16_at(q, i));
            float* p = a.e + row * a.lde + col;
            if (in && a.cols - col >= 8) {
                st8(p, o);
            } else if (in) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col + i < a.cols) p[i] = o[i];
            }
        }
    }
}

// One thread block takes 128 rows by 128 (bf16) or 64 (fp32) columns, 32 KB. The values pass through
// shared memory: for the transposed matrix a thread takes blocks of 32 rows, and its codes go out
// through shared memory as well, so that 64 bytes of a row are written together. VEC: rows' blocks are
// aligned to 32 bytes; they are loaded by 32 bytes and more a lane, and the matrix itself is made from
// registers. Else the values are loaded one by one, consecutive lanes consecutive values: many loads one
// after another (8192 x 1000 bf16, rows of 2000 bytes: the matrix 8.1 us, both forms 10.5; of 1024
// columns 3.6 and 7.6).
//
// Shared memory holds a row as pieces of 16 bytes, which are swapped so that the eight lanes of a store
// (bf16: two rows by four blocks; fp32: a row by eight quarters of blocks) put them into different
// banks; 128 bytes of a row stay together, so that reading along it is free of conflicts too.
template <typename V>
struct MxTile {
    static constexpr int kWide = sizeof(V) == 2 ? 128 : 64;   // columns
    static constexpr int kBlocks = kWide / kMxBlk;
    static constexpr int kParts = kAtomCols / kWide;          // tiles that share an atom of a row form
    static constexpr int kBytes = kAtomRows * kWide * (int)sizeof(V);
    static constexpr int kSmem = kBytes + kWide * 64 + 2 * kAtomBytes;
    static __device__ __forceinline__ int piece(int row, int j) {
        return sizeof(V) == 2 ? j ^ ((j >> 3) & 1) ^ ((row & 1) << 1) : j ^ ((j >> 3) & 1);
    }
    static __device__ __forceinline__ int at(int row, int col) {   // in values
        constexpr int kPer = 16 / (int)sizeof(V);
        return row * kWide + piece(row, col / kPer) * kPer + col % kPer;
    }
};

__device__ __forceinline__ void mx4_kept(const float* tile, int r, int b, Values<float>& v) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float4 t = *reinterpret_cast<const float4*>(tile + MxTile<float>::at(r, 32 * b + 4 * q));
        v.v[4 * q] = t.x;
        v.v[4 * q + 1] = t.y;
        v.v[4 * q + 2] = t.z;
        v.v[4 * q + 3] = t.w;
    }
}
__device__ __forceinline__ void mx4_keep(float* tile, int r, int b, const Values<float>& v) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
        *reinterpret_cast<float4*>(tile + MxTile<float>::at(r, 32 * b + 4 * q)) =
            make_float4(v.v[4 * q], v.v[4 * q + 1], v.v[4 * q + 2], v.v[4 * q + 3]);
}
__device__ __forceinline__ void mx4_kept(const __nv_bfloat16* tile, int r, int b,
                                         Values<__nv_bfloat16>& v) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 t =
            *reinterpret_cast<const uint4*>(tile + MxTile<__nv_bfloat16>::at(r, 32 * b + 8 * q));
        v.w[4 * q] = t.x;
        v.w[4 * q + 1] = t.y;
        v.w[4 * q + 2] = t.z;
        v.w[4 * q + 3] = t.w;
    }
}
__device__ __forceinline__ void mx4_keep(__nv_bfloat16* tile, int r, int b,
                                         const Values<__nv_bfloat16>& v) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(tile + MxTile<__nv_bfloat16>::at(r, 32 * b + 8 * q)) =
            make_uint4(v.w[4 * q], v.w[4 * q + 1], v.w[4 * q + 2], v.w[4 * q + 3]);
}

template <typename T, int FORMS, bool SR, bool VEC, bool RES>
__global__ void __launch_bounds__(kMxThreads) k_mx4_tile(const Mx4QuantArgs a) {
    static_assert(!RES || (FORMS == kMxRows && !VEC), "else k_mx4_rows8");
    after_what_is_ahead();
    using V = typename std::conditional<RES, float, T>::type;   // what the tile holds
    using S = MxTile<V>;
    extern __shared__ __align__(128) uint8_t sm[];
    V* const tile = reinterpret_cast<V*>(sm);
    uint8_t* const codes = sm + S::kBytes;            // [columns][4 blocks][16 bytes]
    uint8_t* const exps = codes + S::kWide * 64;      // an atom, or half of one
    uint8_t* const texps = exps + kAtomBytes;         // the transposed matrix's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t across = a.col_tiles * S::kParts;
    const int64_t ct = blockIdx.x % across, rt = blockIdx.x / across;
    const int64_t r0 = rt * kAtomRows, c0 = ct * S::kWide;
    const T* const x = static_cast<const T*>(a.x) + r0 * a.ld + c0;
    const int rows = (int)min(a.rows - r0, (int64_t)kAtomRows);
    const int cols = (int)max(min(a.cols - c0, (int64_t)S::kWide), (int64_t)0);
    const int64_t pitch = mx4_pitch(a.cols);
    const int blocks = (cols + kMxBlk - 1) / kMxBlk;
    const auto group = [&](int r, int b) { return ((r0 + r) * pitch + c0 / 2) / 4 + b * 4; };
    const auto row_form = [&](int r, int b, const Values<V>& v) -> uint4 {
        uint32_t k = 0;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < rows && b < blocks) {
            w = encode_block<SR>(v, a.key, group(r, b), k);
            *reinterpret_cast<uint4*>(a.c + (r0 + r) * pitch + c0 / 2 + b * 16) = w;
        }
        exps[atom_at(r, b)] = (uint8_t)k;
        return w;
    };
    if constexpr (VEC && sizeof(T) == 2) {
        Values<T> v[2];
        const int b = tid & 3;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = u * 64 + (tid >> 2);
            const int n = r < rows ? min(cols - b * kMxBlk, kMxBlk) : 0;
            const T* p = x + r * a.ld + b * kMxBlk;
            if (n == kMxBlk)
                v[u].load(p);
            else
                v[u].load_some(p, n);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = u * 64 + (tid >> 2);
            if constexpr (FORMS & kMxColumns) mx4_keep(tile, r, b, v[u]);
            if constexpr (FORMS & kMxRows) row_form(r, b, v[u]);
        }
    } else if constexpr (VEC) {
        float v[4][8];
        const int g = tid & 7, c = 8 * g;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = u * 32 + (tid >> 3);
            load8(x + r * a.ld + c, (int64_t)(r < rows ? cols - c : 0), v[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = u * 32 + (tid >> 3), b = g >> 2;
            if constexpr (FORMS & kMxColumns) {
                *reinterpret_cast<float4*>(tile + S::at(r, c)) =
                    make_float4(v[u][0], v[u][1], v[u][2], v[u][3]);
                *reinterpret_cast<float4*>(tile + S::at(r, c + 4)) =
                    make_float4(v[u][4], v[u][5], v[u][6], v[u][7]);
            }
            if constexpr (FORMS & kMxRows) {
                uint32_t k;
                const uint32_t w = encode_quarter<SR>(v[u], a.key, group(r, b) + (g & 3), k);
                if (r < rows && b < blocks)
                    *reinterpret_cast<uint32_t*>(a.c + (r0 + r) * pitch + (c0 + c) / 2) = w;
                if ((g & 3) == 0) exps[atom_at(r, b)] = (uint8_t)k;
            }
        }
    } else {
        constexpr int kPasses = kAtomRows * S::kWide / kMxThreads, kRowParts = S::kWide / 32;
#pragma unroll 4
        for (int i = 0; i < kPasses; ++i) {
            const int r = (i / kRowParts) * kWarps + warp, c = (i % kRowParts) * 32 + lane;
            const bool in = r < rows && c < cols;
            V y = V(0.0f);
            if constexpr (RES) {
                if (in) y = __fadd_rn(ld1(x + r * a.ld + c), a.e[(r0 + r) * a.lde + c0 + c]);
            } else {
                if (in) y = x[r * a.ld + c];
            }
            tile[S::at(r, c)] = y;
        }
        __syncthreads();
        if constexpr (FORMS & kMxRows) {
            const int b = tid % S::kBlocks;
#pragma unroll 1
            for (int r = tid / S::kBlocks; r < kAtomRows; r += kMxThreads / S::kBlocks) {
                Values<V> v;
                mx4_kept(tile, r, b, v);
                const uint4 w = row_form(r, b, v);
                if constexpr (RES) {
                    const uint32_t scale2 = mx4_scale2(exps[atom_at(r, b)]);
                    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint4 q = decode8(c[g], scale2);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v.v[8 * g + i] = __fsub_rn(v.v[8 * g + i], bf16_at(q, i));
                    }
                    mx4_keep(tile, r, b, v);
                }
            }
        }
    }
    if constexpr (FORMS & kMxColumns) {
        const int64_t tpitch = mx4_pitch(a.rows);
        if constexpr (VEC) __syncthreads();
        const int p = tid >> 6;        // the block of rows
        const auto put = [&](auto&& get, uint32_t most, int c) {
            const uint32_t k = mx4_exponent(most);
            *reinterpret_cast<uint4*>(codes + c * 64 + ((p ^ (c >> 1)) & 3) * 16) =
                encode32<SR>(get, k, a.tkey, ((c0 + c) * tpitch + r0 / 2) / 4 + p * 4);
            texps[atom_at(c, p)] = (uint8_t)k;
        };
        if constexpr (sizeof(T) == 4) {
            const int c = tid & 63;
            Values<float> v;
#pragma unroll
            for (int i = 0; i < 32; ++i) v.v[i] = tile[S::at(p * 32 + i, c)];
            put([&](int i) { return v.v[i]; }, v.most(), c);
        } else {
            const int c = (tid & 63) * 2;
            uint32_t w[32];            // two columns
#pragma unroll
            for (int i = 0; i < 32; ++i)
                w[i] = *reinterpret_cast<const uint32_t*>(tile + S::at(p * 32 + i, c));
            uint32_t m[2] = {w[0], w[1]};
#pragma unroll
            for (int i = 2; i < 32; ++i) m[i & 1] = max_magnitude2(m[i & 1], w[i]);
            const uint32_t most = max_magnitude2(m[0], m[1]) & 0x7fff7fffu;
            put([&](int i) { return __uint_as_float(w[i] << 16); }, most << 16, c);
            put([&](int i) { return __uint_as_float(w[i] & 0xffff0000u); }, most & 0xffff0000u, c + 1);
        }
        __syncthreads();
#pragma unroll
        for (int i = tid; i < S::kWide * 4; i += kMxThreads) {
            const int c = i >> 2, q = i & 3;
            const int64_t at = r0 / 2 + q * 16;
            if (c < cols && at < tpitch)
                *reinterpret_cast<uint4*>(a.ct + (c0 + c) * tpitch + at) =
                    *reinterpret_cast<const uint4*>(codes + c * 64 + ((q ^ (c >> 1)) & 3) * 16);
        }
        if (tid < 32) {                // 16 or 8 of an atom's rows of 16 bytes
            uint8_t* to = a.st + ((c0 >> 7) * mx4_atoms(a.rows) + rt) * kAtomBytes + tid * 16;
            const uint8_t* from = texps + tid * 16;
            if constexpr (S::kParts == 1)
                *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
            else
                *reinterpret_cast<uint2*>(to + (ct & 1) * 8) = *reinterpret_cast<const uint2*>(from);
        }
    } else {
        __syncthreads();
    }
    if constexpr (FORMS & kMxRows) {
        uint8_t* to = a.s + (rt * a.col_tiles + ct / S::kParts) * kAtomBytes;
        if constexpr (S::kParts == 1) {
            if (tid >= 32 && tid < 64)
                reinterpret_cast<uint4*>(to)[tid - 32] = reinterpret_cast<const uint4*>(exps)[tid - 32];
        } else {
            if (tid >= 128)
                *reinterpret_cast<uint16_t*>(to + atom_at(tid - 128, (int)(ct & 1) * 2)) =
                    *reinterpret_cast<const uint16_t*>(exps + atom_at(tid - 128, 0));
        }
    }
    if constexpr (RES) {
        constexpr int kPasses = kAtomRows * S::kWide / kMxThreads, kRowParts = S::kWide / 32;
#pragma unroll 4
        for (int i = 0; i < kPasses; ++i) {
            const int r = (i / kRowParts) * kWarps + warp, c = (i % kRowParts) * 32 + lane;
            if (r < rows && c < cols) a.e[(r0 + r) * a.lde + c0 + c] = tile[S::at(r, c)];
        }
    }
}

// ------------------------------------------------------------------------------------------
// reading back

struct Mx4DequantArgs {
    const uint8_t *c, *s;
    void* out;
    int64_t ld, rows, cols, col_tiles;
    int32_t segments, segment, rows_per;   // as in Mx4QuantArgs, but of the blocks that there are
    uint32_t magic;                        // (0 for one block)
};

// To fp32 whose blocks are aligned to 32 bytes: eight values a thread, contiguous in a warp (8192 x
// 8192: 50 us; a block a thread 63).
__global__ void __launch_bounds__(kMxThreads) k_mx4_dequantize8(const Mx4DequantArgs a) {
    after_what_is_ahead();
    const int blocks = (int)mx4_blocks(a.cols), g = threadIdx.x & 3;
    const int64_t pitch = mx4_pitch(a.cols);
    MxPlace t[kMxUnits];
    uint32_t c[kMxUnits], k[kMxUnits];
#pragma unroll
    for (int u = 0; u < kMxUnits; ++u) {
        t[u] = mx4_place((int)threadIdx.x / 4 + u * (kMxThreads / 4), blocks, a.segments, a.segment,
                         a.rows_per, a.magic, a.rows);
        c[u] = k[u] = 0;
        if (t[u].in) {
            c[u] = *reinterpret_cast<const uint32_t*>(a.c + t[u].row * pitch + t[u].b * 16 + g * 4);
            k[u] = a.s[((t[u].row >> 7) * a.col_tiles + (t[u].b >> 2)) * kAtomBytes +
                       atom_at((int)(t[u].row & 127), t[u].b & 3)];
        }
    }
#pragma unroll
    for (int u = 0; u < kMxUnits; ++u) {
        if (!t[u].in) continue;
        const uint4 v = decode8(c[u], mx4_scale2(k[u]));
        const int64_t col = (int64_t)t[u].b * kMxBlk + 8 * g;
        float* out = static_cast<float*>(a.out) + t[u].row * a.ld + col;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = bf16_at(v, i);
        if (a.cols - col >= 8) {
            st8(out, o);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < a.cols) out[i] = o[i];
        }
    }
}

// A thread a block. VEC (bf16): out's blocks are aligned to 32 bytes. Else the values go through shared memory
// (a warp's 32 blocks, which may be of several rows) and out by 16 bytes a lane from the first such
// address on, because a store instruction takes as long for less (1024 x 30522 to bf16: by two bytes a
// lane 94 us, by four 38).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads) k_mx4_dequantize(const Mx4DequantArgs a) {
    after_what_is_ahead();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (int)mx4_blocks(a.cols);
    const MxPlace t = mx4_place(tid, blocks, a.segments, a.segment, a.rows_per, a.magic, a.rows);
    const int64_t row = t.row;
    const int b = t.b;
    const bool in = t.in;
    uint4 c = make_uint4(0, 0, 0, 0);
    uint32_t scale2 = 0;
    if (in) {
        c = *reinterpret_cast<const uint4*>(a.c + row * mx4_pitch(a.cols) + b * 16);
        scale2 = mx4_scale2(a.s[((row >> 7) * a.col_tiles + (b >> 2)) * kAtomBytes +
                                atom_at((int)(row & 127), b & 3)]);
    }
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint4 v[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) v[g] = decode8(w[g], scale2);
    T* const out = static_cast<T*>(a.out) + row * a.ld + (int64_t)b * kMxBlk;
    const int n = in ? (int)min(a.cols - (int64_t)b * kMxBlk, (int64_t)kMxBlk) : 0;
    if (VEC && n == kMxBlk) {
#pragma unroll
        for (int g = 0; g < 4; g += 2)
            asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(v[g].x),
                         "r"(v[g].y), "r"(v[g].z), "r"(v[g].w), "r"(v[g + 1].x), "r"(v[g + 1].y),
                         "r"(v[g + 1].z), "r"(v[g + 1].w), "l"(out + 8 * g)
                         : "memory");
    } else if (VEC) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) st1(out + i, bf16_at(v[i >> 3], i & 7));
    } else {
        // block l of the warp: 16 words of two values, word j at l * 16 + (j ^ l % 16)
        __shared__ uint32_t values[kWarps][32 * 16];
        uint32_t* const mine = values[warp];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const uint32_t u[4] = {v[g].x, v[g].y, v[g].z, v[g].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[lane * 16 + ((4 * g + i) ^ (lane & 15))] = u[i];
        }
        // runs of blocks of one row: this lane begins one if the lane before has another row
        const uint32_t low = (uint32_t)row;
        const uint32_t before = __shfl_up_sync(kFull, low, 1);
        uint32_t starts = __ballot_sync(kFull, in && (lane == 0 || before != low));
        const uint32_t there = __ballot_sync(kFull, in);
        __syncwarp();
        const uint64_t at = reinterpret_cast<uint64_t>(out);
        while (starts != 0) {
            const int l0 = __ffs(starts) - 1;
            starts &= starts - 1;
            const int l1 = starts != 0 ? __ffs(starts) - 1 : 32 - __clz(there);
            T* const o = reinterpret_cast<T*>(__shfl_sync(kFull, at, l0));
            const int m = (l1 - 1 - l0) * kMxBlk + __shfl_sync(kFull, n, l1 - 1);   // values of the run
            const auto word = [&](int j) { return mine[(l0 * 16 + j) ^ ((l0 + (j >> 4)) & 15)]; };
            const auto one = [&](int i) {
                const uint32_t x = word(i >> 1);
                return __uint_as_float((i & 1) ? x & 0xffff0000u : x << 16);
            };
            // whole 16 bytes from the first such address on, and what is before and behind them
            constexpr int kPer = 16 / (int)sizeof(T);
            const int head = min(m, (int)((16 - (reinterpret_cast<uint64_t>(o) & 15)) & 15) / (int)sizeof(T));
            const int whole = (m - head) / kPer;
            for (int j = lane; j < whole; j += 32) {
                const int i = head + j * kPer;
                if constexpr (sizeof(T) == 4) {
                    float4 f;
                    f.x = one(i);
                    f.y = one(i + 1);
                    f.z = one(i + 2);
                    f.w = one(i + 3);
                    *reinterpret_cast<float4*>(o + i) = f;
                } else {
                    uint32_t w[5];
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[q] = word((i >> 1) + q);
                    w[4] = (i & 1) ? word((i >> 1) + 4) : 0u;
                    const int shift = (i & 1) * 16;
                    *reinterpret_cast<uint4*>(o + i) = make_uint4(
                        __funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift),
                        __funnelshift_r(w[2], w[3], shift), __funnelshift_r(w[3], w[4], shift));
                }
            }
            const int rest = m - whole * kPer;                 // values before and behind
            if (lane < rest) {
                const int i = lane < head ? lane : lane + whole * kPer;
                st1(o + i, one(i));
            }
        }
    }
}

}  // namespace onebit
