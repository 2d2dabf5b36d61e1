// kernels_mx4.cuh -- matrices in microscaled 4-bit floating point for B200 (sm_100a): quantising,
// reading back, and the product of two of them on the tensor cores.
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

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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
// code. w: the random word of the group of eight. Instructions bound it, 14 a value: the integer ones
// that make the random bits most of all.
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

// Eight values to codes in a block of exponent k; w: the random word.
template <bool SR>
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t k, uint32_t w) {
    float z[8];
    uint32_t c;
    if constexpr (SR) {
        // one factor where fp32 has it, 2^(1 - k)
        if (k <= 127u) {
            const float f = k == 0u ? 2.0f : __uint_as_float((128u - k) << 23);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = __fmul_rz(v[i], f);
        } else {
            const float inv = mx4_inverse(k);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = __fmul_rz(v[i] * inv, 0x1p-126f);
        }
        c = encode8_stochastic(z, w);
    } else {
        const float inv = mx4_inverse(k);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = v[i] * inv;
        c = encode8_nearest(z);
    }
    return k == kMxNan ? 0u : c;
}

// Largest magnitudes by their patterns: any NaN is above infinity.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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
        uint32_t m[2] = {w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu};
#pragma unroll
        for (int i = 2; i < 16; ++i) m[i & 1] = max_u16x2(m[i & 1], w[i] & 0x7fff7fffu);
        const uint32_t x = max_u16x2(m[0], m[1]);
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
    const uint32_t kh = SR ? key + (uint32_t)(G >> 32) * kGolden : 0u;
    uint32_t w[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = get(8 * g + i);
        w[g] = encode8<SR>(v, k, SR ? mix32((uint32_t)G + g + kh) : 0u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// The same with the exponent that the block takes.
template <bool SR, typename V>
__device__ __forceinline__ uint4 encode_block(const V& v, uint32_t key, int64_t G, uint32_t& k) {
    k = mx4_exponent(v.most());
    return encode32<SR>([&](int i) { return v.get(i); }, k, key, G);
}

// Eight codes (a word) as bf16 values times a power of two: both bytes of a magnitude come from a
// table of eight, the signs go on top. Exact: bf16 holds every such value.
__device__ __forceinline__ uint4 decode8(uint32_t c, uint32_t scale2) {
    uint32_t o[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t x = h == 0 ? c : c >> 16, sel = x & 0x7777u;
        const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, sel);
        const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, sel);
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
    return encode8<SR>(v, k, SR ? group_word(key, G) : 0u);
}

constexpr int kMxUnits = 2;

template <typename T, bool SR, bool RES>
__global__ void __launch_bounds__(kMxThreads) k_mx4_rows8(const Mx4QuantArgs a) {
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
// registers. Else the values are loaded one by one, consecutive lanes consecutive values.
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
            uint32_t m[2] = {w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu};
#pragma unroll
            for (int i = 2; i < 32; ++i) m[i & 1] = max_u16x2(m[i & 1], w[i] & 0x7fff7fffu);
            const uint32_t most = max_u16x2(m[0], m[1]);
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
// (a warp's 32 blocks, which may be of several rows) and out by consecutive lanes; bf16 by pairs from an
// even address on, because stores of two bytes a lane are slow (1024 x 30522: 94 us).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads) k_mx4_dequantize(const Mx4DequantArgs a) {
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
        __syncwarp();
        const auto value = [&](int l, int i) -> uint32_t {
            return (mine[l * 16 + ((i >> 1) ^ (l & 15))] >> (16 * (i & 1))) & 0xffffu;
        };
        const uint64_t at = reinterpret_cast<uint64_t>(out);
#pragma unroll 1
        for (int l = 0; l < 32; l += 2) {
            // two blocks at a time: half a warp each
            const int from = l + (lane >> 4), half = lane & 15;
            const uint64_t p = __shfl_sync(kFull, at, from);
            const int m = __shfl_sync(kFull, n, from);
            if constexpr (sizeof(T) == 4) {
                float* o = reinterpret_cast<float*>(p);
#pragma unroll
                for (int i = half; i < 32; i += 16)
                    if (i < m) o[i] = __uint_as_float(value(from, i) << 16);
            } else {
                uint16_t* o = reinterpret_cast<uint16_t*>(p);
                const int odd = (int)(p >> 1) & 1, i = 2 * half + odd;  // the pair from value i on
                if (i + 1 < m)
                    *reinterpret_cast<uint32_t*>(o + i) = value(from, i) | value(from, i + 1) << 16;
                else if (i < m)
                    o[i] = (uint16_t)value(from, i);
                if (odd && half == 0 && m > 0) o[0] = (uint16_t)value(from, 0);
            }
        }
    }
}

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
// That halves what each reads of a.
//
// Warps: 0 loads (TMA), 1 issues the products, 2 to 5 write out, 6 to 9 move the exponents from shared
// to tensor memory (each its quarter of the lanes; every quarter holds all of them). The tensor cores'
// own copies (tcgen05.cp) wait for the products before them and hold up those behind: 75 clocks an
// atom, six for every four products (8192^3: 358 us with them).

constexpr int kMmThreads = 320;
constexpr int kMmLanes = 128;             // rows of b in a block's part of a tile
constexpr int kStageCols = 256;
constexpr int kExpBuffers = 4;            // stages whose exponents are in tensor memory
constexpr uint32_t kMmTimeout = 1u;
constexpr int kOutBytes = 2048;           // written out at a time: 32 columns of out by 32 rows (bf16)
constexpr int kOutRows32 = 16;            // ... or by 16 (fp32)

__device__ uint32_t g_mx4_status;

template <int TM, bool PAIR, bool SPLIT>
struct MmTile {
    static constexpr int kGroup = PAIR ? 2 : 1;
    static constexpr int kARows = TM / kGroup;                // rows of a that a block loads
    static constexpr int kHalves = TM > 128 ? 2 : 1;          // atoms of a's exponents across
    static constexpr int kB = kMmLanes * 128, kA = kARows * 128;  // bytes of codes in a stage
    static constexpr int kSB = 2 * kAtomBytes, kSA = 2 * kHalves * kAtomBytes;
    static constexpr int kStage = kB + kA + kSB + kSA;
    // Behind the stages: what is written out (two buffers for each of four warps), or the sums of a
    // split tile from the other blocks, [block][its rows][128].
    static constexpr int kParts = SPLIT ? (TM + 8) * kMmLanes * 4 : 4 * 2 * kOutBytes;
    static constexpr int kBarriers = 512;
    static constexpr int kMost = (227 * 1024 - kBarriers - kParts) / kStage;
    static constexpr int kStages = kMost < 8 ? kMost : 8;
    static constexpr int kSmem = kStages * kStage + kParts + kBarriers;
    static_assert(kStages >= kExpBuffers, "the exponents' buffers are freed with the stages");
    // Tensor memory: two accumulators and the exponents. Two of 256 columns leave no room: they
    // overlap by 96 columns, which are read first.
    static constexpr int kOverlap = TM == 256 ? 96 : 0;
    static constexpr int kSecond = TM - kOverlap;
    static constexpr int kExp = kSecond + TM;
    static constexpr int kExpCols = 8 + 8 * kHalves;
    static constexpr int kNeed = kExp + kExpBuffers * kExpCols;
    static constexpr int kColumns = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static_assert(kNeed <= 512, "tensor memory");
    static constexpr int kChunk = TM < 32 ? TM : 32;          // columns taken out at a time
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
};

__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, int x, int y,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
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

// Arrive on a barrier of a pair's first block. What the arrival announces are finished copies (TMA) and
// stores to tensor memory, which the tensor cores of the arriving block's own SM read, and no plain
// stores: the arrival needs no fence of the cluster's scope (with one, 8192^3 takes 423 us, without
// 240).
template <bool PAIR>
__device__ __forceinline__ void pair_arrive(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                         cluster_addr(smem_addr(bar), 0))
                     : "memory");
    else
        mbar_arrive(bar);
}
// One lane of a warp that runs together: the compiler keeps what such a branch's instructions take in
// uniform registers, which a branch on the lane's number does not let it (see k_mx4_matmul).
__device__ __forceinline__ bool elect() {
    uint32_t yes;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(yes));
    return yes != 0;
}

// What a warp writes out: buffers in shared memory, and where they go.
struct OutWarp {
    const CUtensorMap* map;
    uint8_t* buf;              // two of kOutBytes
    int n0;                    // the warp's first column of out
    int lane;
    int count;                 // buffers filled
};

// The next buffer, once the copy out of it is over.
__device__ __forceinline__ uint8_t* out_buffer(OutWarp& w) {
    if (w.lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    return w.buf + (w.count++ & 1) * kOutBytes;
}
// Copy a buffer out, its first row being `row`; the map leaves out what lies behind the edges.
__device__ __forceinline__ void out_copy(const OutWarp& w, const uint8_t* buf, int row) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (w.lane == 0) {
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(w.map),
            "r"(w.n0), "r"(row), "r"(smem_addr(buf))
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
// each has eight columns of a row 61.)
template <int N, typename OT>
__device__ __forceinline__ void put_chunk(const Mx4MatmulArgs& p, OutWarp& w, float* v, int row,
                                          int rows) {
    const int lane = w.lane;
    if (rows <= 0 || w.n0 >= p.n) return;
    if constexpr (sizeof(OT) == 4) {
        float* const out = static_cast<float*>(p.out) + (int64_t)row * p.ld + w.n0 + lane;
        const bool in = w.n0 + lane < p.n;
        constexpr int kB = N < kOutRows32 ? N : kOutRows32;
#pragma unroll
        for (int h = 0; h < N; h += kB) {
            if (p.accumulate) {
                float o[kB];
#pragma unroll
                for (int j = 0; j < kB; ++j)
                    o[j] = in && h + j < rows ? out[(h + j) * p.ld] : 0.0f;
#pragma unroll
                for (int j = 0; j < kB; ++j) v[h + j] += o[j];
            }
            if (p.tma) {
                if (h < rows) {
                    uint8_t* buf = out_buffer(w);
#pragma unroll
                    for (int j = 0; j < kB; ++j) reinterpret_cast<float*>(buf)[j * 32 + lane] = v[h + j];
                    out_copy(w, buf, row + h);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kB; ++j)
                    if (in && h + j < rows) out[(h + j) * p.ld] = v[h + j];
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
            out_copy(w, buf, row);
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
    uint64_t* const done = empty + S::kStages;      // [2] an accumulator is complete
    uint64_t* const drained = done + 2;             // [2] ... and read as far as the next needs
    uint64_t* const last = drained + 2;
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(last + 1);
    const int warp = (int)__shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(ready + i, 4 * S::kGroup);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(done + i, 1);
            mbar_init(drained + i, 4 * S::kGroup);
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
                if (!(ok = mbar_wait_bounded(empty + stage, phase ^ 1))) break;
                uint8_t* s = sm + stage * S::kStage;
                if (elect()) {
                    mbar_arrive_expect_tx(full + stage, S::kStage);
                    tma_tile(s, &maps.b, k * 128, brow * kMmLanes, full + stage);
                    tma_tile(s + S::kB, &maps.a, k * 128, tm * TM + bank * S::kARows, full + stage);
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
        if (!ok && lane == 0) {  // leave no copy in flight behind
            atomicOr(&g_mx4_status, kMmTimeout);
            for (int64_t f = filled > S::kStages ? filled - S::kStages : 0; f < filled; ++f)
                mbar_wait_bounded(full + f % S::kStages, (uint32_t)(f / S::kStages) & 1);
        }
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
                !(ok = mbar_wait_bounded(drained + (before & 1), (uint32_t)(before >> 1) & 1)))
                break;
            tc_fence_after();
            for (int k = k0; k < k1; ++k, ++c) {
                if (!(ok = mbar_wait_bounded(ready + stage, phase))) break;
                tc_fence_after();
                const uint32_t s = smem_addr(sm + stage * S::kStage);
                const uint32_t eb = tmem + S::kExp + (c % kExpBuffers) * S::kExpCols, ea = eb + 8;
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
        if (!ok && lane == 0) {
            atomicOr(&g_mx4_status, kMmTimeout);
            tc_commit<PAIR>(last);
            mbar_wait_bounded(last, 0);
        }
    } else if (warp >= 2 && warp < 6) {
        const int quad = warp & 3;
        OutWarp w{&maps.out, reinterpret_cast<uint8_t*>(parts) + quad * 2 * kOutBytes, 0, lane, 0};
        int i = 0;
        for (int t = first; t < tiles && ok; t += hop, ++i) {
            int tm, tn;
            place(t, tm, tn);
            const int buf = i & 1;
            if (!(ok = mbar_wait_bounded(done + buf, (uint32_t)(i >> 1) & 1))) break;
            tc_fence_after();
            const uint32_t d = tmem + buf * S::kSecond + ((uint32_t)(quad * 32) << 16);
            const int64_t m0 = (int64_t)tm * TM;
            const int rows = (int)min((int64_t)TM, p.m - m0);
            w.n0 = (tn * S::kGroup + bank) * kMmLanes + quad * 32;
            constexpr int kC = S::kChunk;
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
                __syncwarp();
                tc_load<kC>(d, v);
                tc_load_wait<kC>(v);
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    const uint32_t at = __shfl_sync(kFull, to_row, j);
                    if (j < rows) cluster_store(at + (quad * 32 + lane) * 4, v[j]);
                }
            } else if constexpr (S::kOverlap > 0) {
                // what the accumulators share first: the last columns of the first, the first of the
                // second
                constexpr int kFirst = S::kOverlap / kC, kRest = TM / kC - kFirst;
                const int at = buf == 0 ? kRest * kC : 0, rest = buf == 0 ? 0 : S::kOverlap;
                float v[kFirst * kC];
                __syncwarp();
#pragma unroll
                for (int u = 0; u < kFirst; ++u) take_chunk<kC, OT>(d + at + u * kC, v + u * kC);
                tc_load_wait<kFirst * kC>(v);
                read_done();
#pragma unroll
                for (int u = 0; u < kFirst; ++u)
                    put_chunk<kC, OT>(p, w, v + u * kC, (int)m0 + at + u * kC, rows - at - u * kC);
#pragma unroll 1
                for (int j0 = rest; j0 < rest + kRest * kC && j0 < rows; j0 += kC) {
                    __syncwarp();
                    take_chunk<kC, OT>(d + j0, v);
                    tc_load_wait<kC>(v);
                    put_chunk<kC, OT>(p, w, v, (int)m0 + j0, rows - j0);
                }
            } else {
#pragma unroll 1
                for (int j0 = 0; j0 < TM; j0 += kC) {
                    float v[kC];
                    __syncwarp();
                    take_chunk<kC, OT>(d + j0, v);
                    tc_load_wait<kC>(v);
                    if (j0 + kC == TM) read_done();
                    put_chunk<kC, OT>(p, w, v, (int)m0 + j0, rows - j0);
                }
            }
        }
        if (!SPLIT && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok && lane == 0) atomicOr(&g_mx4_status, kMmTimeout);
    } else if (warp >= 6) {
        int stage = 0, c = 0;
        uint32_t phase = 0;
        for (int t = first; t < tiles && ok; t += hop) {
            int tm, tn;
            place(t, tm, tn);
            // narrow tiles: the word of the tile's first rows (32 of the atom's 128 a word) comes first,
            // since the tensor cores take exponents from even columns on only
            const int sub = TM < kAtomRows ? tm * TM % kAtomRows / 32 : 0;
            for (int k = k0; k < k1; ++k, ++c) {
                // the products that read this buffer before are done, and the stage is there
                const int b = c - kExpBuffers;
                if (b >= 0 && !(ok = mbar_wait_bounded(empty + b % S::kStages,
                                                       (uint32_t)(b / S::kStages) & 1)))
                    break;
                if (!(ok = mbar_wait_bounded(full + stage, phase))) break;
                const uint4* e = reinterpret_cast<const uint4*>(sm + stage * S::kStage + S::kB + S::kA) +
                                 lane;
                const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + S::kExp +
                                    (c % kExpBuffers) * S::kExpCols;
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

}  // namespace onebit
