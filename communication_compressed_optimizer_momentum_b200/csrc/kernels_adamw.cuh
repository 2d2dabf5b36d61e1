// kernels_adamw.cuh -- AdamW over a list of tensors for B200 (sm_100a): the step with 32-bit and
// with 8-bit states, the global gradient norm, and the conversion of the 8-bit states.
//
// Work unit: a BLOCK of kBlk = 256 consecutive elements of one tensor, owned by one warp, eight
// elements a lane. The states of all tensors lie in one flat vector in which every tensor begins
// at a block boundary, so a block of a tensor is a block of the state. The tensors' addresses
// travel in the kernel parameters (TensorTable, up to 30 KB), so a call queues exactly one launch
// and keeps nothing: no table in device memory to upload, to go stale, or to be shared.
//
// All of it streams HBM once; nothing is a contraction.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.cuh"

namespace onebit {

constexpr int kBlk = 256;             // elements of a state block
constexpr int kBlkLane = kBlk / 32;   // of one lane
constexpr uint32_t kGolden = 0x9E3779B9u;
constexpr uint16_t kTabVec = 0x8000u;  // TensorTable::last: all addresses take 16-byte accesses

// The tensors of one launch (empty ones left out).
template <int N>
struct TensorTable {
    int32_t n;
    uint32_t nblk;           // blocks of all tensors
    int64_t blk0;            // state block of the first
    uint32_t first[N + 1];   // first block of each tensor, counted from blk0
    uint16_t last[N];        // elements in its last block (1..256), kTabVec
    void* p[N];              // parameters
    const void* g[N];        // gradients
    void* c[N];              // bf16 copies (or null)
    double wd[N];            // weight decay
};

// Device-side progress of one optimizer: ONEBIT_ADAMW_CTL_BYTES, all zero at the start.
struct StepCtl {
    int64_t t;         // steps taken
    int64_t skipped;   // steps left out because the gradient scale was not finite
    double c1, c2;     // 1 - beta^t, kept as the running mean of ones: c = beta c + (1 - beta)
    uint32_t ticket;   // blocks of the running launch that are done
    uint32_t pad[7];
};

struct StepArgs {
    double lr, beta1, beta2, omb1, omb2;
    const double* lr_dev;    // overrides lr (or null)
    const float* scale;      // factor on every gradient (or null)
    float eps;
    int32_t bias;            // bias correction on
    int32_t advance;         // this launch is the step's last: count it
    uint64_t seed;           // 8-bit states: stochastic rounding
    StepCtl* ctl;
    float* m;                // 32-bit states
    float* v;
    uint8_t* mc;             // 8-bit states: codes and block exponents
    uint8_t* vc;
    uint8_t* mk;
    uint8_t* vk;
};

// ------------------------------------------------------------------------------------------
// eight consecutive values of a lane

__device__ __forceinline__ void ld8(const float* p, float (&o)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}

__device__ __forceinline__ void st8(float* p, const float (&o)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float (&o)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void st8(__nv_bfloat16* p, const float (&o)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A lane's eight elements of a block: consecutive ones (VEC: a whole block whose addresses take
// 16-byte accesses), else every 32nd, so that a warp's accesses are contiguous at any alignment.
template <bool VEC>
__device__ __forceinline__ int elem(int lane, int i) {
    return VEC ? lane * kBlkLane + i : i * 32 + lane;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load(const T* p, int lane, int len, float (&o)[8]) {
    if constexpr (VEC) {
        ld8(p + lane * kBlkLane, o);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = i * 32 + lane < len ? ld1(p + i * 32 + lane) : 0.0f;
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store(T* p, int lane, int len, const float (&o)[8]) {
    if constexpr (VEC) {
        st8(p + lane * kBlkLane, o);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * 32 + lane < len) st1(p + i * 32 + lane, o[i]);
    }
}

// ------------------------------------------------------------------------------------------
// the walk over the tensors

// The tensor that block b belongs to.
template <int N>
__device__ __forceinline__ int tensor_of(const TensorTable<N>& t, uint32_t b) {
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b >= t.first[mid]) lo = mid; else hi = mid;
    }
    return lo;
}

// The step's scalars. fp64, rounded once.
struct StepScalars {
    double lr;
    float step, r2, scale;
    float b1, omb1, b2, omb2, eps;
    bool skip;
};

__device__ __forceinline__ double mean_of_ones(double c, double beta, double omb) {
    return __dadd_rn(__dmul_rn(beta, c), omb);
}

__device__ __forceinline__ StepScalars step_scalars(const StepArgs& a) {
    StepScalars s;
    s.scale = a.scale ? *a.scale : 1.0f;
    s.lr = a.lr_dev ? *a.lr_dev : a.lr;
    double c1 = 1.0, c2 = 1.0;
    if (a.bias) {
        c1 = mean_of_ones(a.ctl->c1, a.beta1, a.omb1);
        c2 = mean_of_ones(a.ctl->c2, a.beta2, a.omb2);
    }
    s.step = (float)(s.lr / c1);
    s.r2 = (float)(1.0 / sqrt(c2));
    s.b1 = (float)a.beta1;
    s.omb1 = (float)a.omb1;
    s.b2 = (float)a.beta2;
    s.omb2 = (float)a.omb2;
    s.eps = a.eps;
    s.skip = !isfinite(s.scale);
    return s;
}

// Count the step once every block of its last launch is done with the scalars.
__device__ __forceinline__ void step_done(const StepArgs& a, bool skip) {
    if (!a.advance) return;
    __syncthreads();
    if (threadIdx.x != 0) return;
    StepCtl* c = a.ctl;
    __threadfence();
    if (atomicAdd(&c->ticket, 1u) != gridDim.x - 1) return;
    c->ticket = 0;
    if (skip) {
        c->skipped += 1;
    } else {
        c->t += 1;
        c->c1 = mean_of_ones(c->c1, a.beta1, a.omb1);
        c->c2 = mean_of_ones(c->c2, a.beta2, a.omb2);
    }
}

//   m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2
__device__ __forceinline__ void adam_moments(const StepScalars& s, float g, float& m, float& v) {
    const float gs = __fmul_rn(g, s.scale);
    m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.omb1, gs));
    v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(s.omb2, __fmul_rn(gs, gs)));
}

//   p = p (1 - lr wd) - (lr / c1) * m / (sqrt(v) / sqrt(c2) + eps)
__device__ __forceinline__ float adam_param(const StepScalars& s, float keep, float p, float m,
                                            float v) {
    const float den = __fadd_rn(__fmul_rn(__fsqrt_rn(v), s.r2), s.eps);
    return __fsub_rn(__fmul_rn(p, keep), __fmul_rn(s.step, __fdiv_rn(m, den)));
}

// ------------------------------------------------------------------------------------------
// 32-bit states

template <bool VEC, typename PT, typename GT>
__device__ __forceinline__ void adamw_block(const StepScalars& s, float keep, PT* p, const GT* g,
                                            __nv_bfloat16* c, float* m, float* v, int lane,
                                            int len) {
    float pv[8], gv[8], mv[8], vv[8];
    load<VEC>(g, lane, len, gv);
    load<VEC>(m, lane, len, mv);
    load<VEC>(v, lane, len, vv);
    load<VEC>(p, lane, len, pv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        adam_moments(s, gv[i], mv[i], vv[i]);
        pv[i] = adam_param(s, keep, pv[i], mv[i], vv[i]);
    }
    store<VEC>(m, lane, len, mv);
    store<VEC>(v, lane, len, vv);
    store<VEC>(p, lane, len, pv);
    if (c) store<VEC>(c, lane, len, pv);
}

template <typename PT, typename GT, int N>
__global__ void __launch_bounds__(kThreads, 4)
k_adamw(const __grid_constant__ TensorTable<N> t, const StepArgs a) {
    const StepScalars s = step_scalars(a);
    const int lane = threadIdx.x & 31;
    if (!s.skip) {
        uint32_t b = blockIdx.x * kWarps + (threadIdx.x >> 5);
        const uint32_t hop = gridDim.x * kWarps;
        int i = tensor_of(t, b);
        float keep = 0.0f;
        int known = -1;
        for (; b < t.nblk; b += hop) {
            while (b >= t.first[i + 1]) ++i;
            if (i != known) {
                keep = (float)(1.0 - s.lr * t.wd[i]);
                known = i;
            }
            const int64_t e = (int64_t)(b - t.first[i]) * kBlk, se = (t.blk0 + b) * kBlk;
            const int len = b + 1 == t.first[i + 1] ? t.last[i] & 0x1ff : kBlk;
            PT* p = static_cast<PT*>(t.p[i]) + e;
            const GT* g = static_cast<const GT*>(t.g[i]) + e;
            __nv_bfloat16* c = static_cast<__nv_bfloat16*>(t.c[i]);
            if (c) c += e;
            if (len == kBlk && (t.last[i] & kTabVec))
                adamw_block<true>(s, keep, p, g, c, a.m + se, a.v + se, lane, len);
            else
                adamw_block<false>(s, keep, p, g, c, a.m + se, a.v + se, lane, len);
        }
    }
    step_done(a, s.skip);
}

// ------------------------------------------------------------------------------------------
// 8-bit states
//
// One exponent k for a block of 256 elements of m (and one for v): the block's values are
// small floats below a common power of two,
//   m: sign, 4 exponent bits, 3 mantissa bits;   v: 5 exponent bits, 3 mantissa bits, no sign,
// the largest code being 1.875 * 2^(k-127). The scale is a power of two, so scaling is exact and
// costs the format no precision: z = |x| * 2^(TOP - k) puts the block's largest value at exponent
// field TOP of an fp32 number, and the code is then simply the upper bits of z's pattern, subnormal
// codes included (they line up with fp32's own subnormals; nothing flushes to zero here).
// A block that holds an infinity or a NaN gets k = 255 and reads back as NaN.
//
// Rounding in the step is stochastic: beta2 = 0.999 moves v by at most about 0.1 % a step, below
// half a step of a 3-bit mantissa, so rounding to nearest would freeze v; rounding up with the
// probability of the remainder keeps the mean of v (and m) that of the exact recurrence. A
// positive v never gets code 0, so a denominator is at least 2^-16.5 of its block's largest, about
// the ratio below which m reads as 0.

constexpr int kTopM = 15, kTopV = 31;
constexpr uint32_t kExpNan = 255u;

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The block's exponent: the smallest window whose largest code holds the block's largest
// magnitude (as fp32 patterns, which order like the magnitudes; infinities and NaN end at 255).
__device__ __forceinline__ uint32_t block_exponent(uint32_t largest) {
    return min((largest + 0xFFFFFu) >> 23, kExpNan);
}

// Factors of a block: 2^(TOP - k) in two exact steps where one is out of fp32's range (k > 130,
// magnitudes above 2^4 -- rare, and the second factor is 1 elsewhere).
template <int TOP>
__device__ __forceinline__ void encode_factors(uint32_t k, float& f1, float& f2) {
    const int far = max((int)k - 130, 0);
    f1 = pow2(-far);
    f2 = pow2(TOP - (int)k + far);
}
template <int TOP>
__device__ __forceinline__ void decode_factors(uint32_t k, float& f1, float& f2) {
    const int far = max((int)k - 130, 0);
    f1 = pow2((int)k - far - TOP);
    f2 = k == kExpNan ? __int_as_float(0x7fffffff) : pow2(far);
}

template <int TOP>
__device__ __forceinline__ float decode_value(uint32_t code, float f1, float f2) {
    if constexpr (TOP == kTopM) {
        const float z = __uint_as_float((code & 127u) << 20);
        const float x = __fmul_rn(__fmul_rn(z, f1), f2);
        return __uint_as_float(__float_as_uint(x) | ((code & 128u) << 24));
    } else {
        return __fmul_rn(__fmul_rn(__uint_as_float(code << 20), f1), f2);
    }
}

// `add` is 20 random bits, or what rounds to nearest even.
template <int TOP>
__device__ __forceinline__ uint32_t encode_bits(float x, float f1, float f2) {
    return __float_as_uint(__fmul_rn(__fmul_rn(fabsf(x), f1), f2));
}
template <int TOP>
__device__ __forceinline__ uint32_t encode_value(float x, uint32_t z, uint32_t add) {
    uint32_t c = (z + add) >> 20;
    if constexpr (TOP == kTopM)
        c |= (__float_as_uint(x) >> 24) & 128u;
    else
        c = max(c, min(__float_as_uint(x), 1u));
    return c;
}

// 32 random bits from 32: two rounds of xor-shift and odd multiplication.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x9016D2F5u;
    x ^= x >> 15;
    x *= 0x314549A1u;
    return x ^ (x >> 16);
}
// The step's key, and a group's: state elements 8G .. 8G+7.
__device__ __forceinline__ uint32_t step_key(uint64_t seed, int64_t t) {
    return mix32(mix32(mix32((uint32_t)seed + kGolden) ^ (uint32_t)(seed >> 32)) + (uint32_t)t);
}
__device__ __forceinline__ uint32_t group_word(uint32_t key, int64_t G) {
    return mix32((uint32_t)G + key + (uint32_t)(G >> 32) * kGolden);
}
// Element j of a group: 16 random bits for v in the lower half, 16 for m in the upper.
__device__ __forceinline__ uint32_t element_bits(uint32_t w, int j) {
    uint32_t x = w + (uint32_t)(j + 1) * kGolden;
    x ^= x >> 15;
    x *= 0x8A8866C7u;
    return x ^ (x >> 16);
}

template <bool VEC>
__device__ __forceinline__ void load_codes(const uint8_t* p, int lane, int len, uint32_t (&o)[8]) {
    if constexpr (VEC) {
        const uint2 w = *reinterpret_cast<const uint2*>(p + lane * kBlkLane);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = i * 32 + lane < len ? p[i * 32 + lane] : 0u;
    }
}
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, int lane, int len, const uint32_t (&o)[8]) {
    if constexpr (VEC) {
        uint2 w;
        w.x = o[0] | o[1] << 8 | o[2] << 16 | o[3] << 24;
        w.y = o[4] | o[5] << 8 | o[6] << 16 | o[7] << 24;
        *reinterpret_cast<uint2*>(p + lane * kBlkLane) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * 32 + lane < len) p[i * 32 + lane] = (uint8_t)o[i];
    }
}

template <int TOP, bool VEC>
__device__ __forceinline__ void load_state(const uint8_t* codes, uint32_t k, int lane, int len,
                                           float (&x)[8]) {
    uint32_t q[8];
    load_codes<VEC>(codes, lane, len, q);
    float f1, f2;
    decode_factors<TOP>(k, f1, f2);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = decode_value<TOP>(q[i], f1, f2);
}

// Encode a block's values (elements past len are 0); add[i] is used where STOCHASTIC.
template <int TOP, bool VEC, bool STOCHASTIC>
__device__ __forceinline__ void store_state(uint8_t* codes, uint8_t* exps, int lane, int len,
                                            const float (&x)[8], const uint32_t (&add)[8]) {
    uint32_t largest = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
        if (VEC || i * 32 + lane < len) largest = max(largest, a);
    }
    const uint32_t k = block_exponent(__reduce_max_sync(kFull, largest));
    float f1, f2;
    encode_factors<TOP>(k, f1, f2);
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t z = encode_bits<TOP>(x[i], f1, f2);
        const uint32_t r = STOCHASTIC ? add[i] : 0x7FFFFu + ((z >> 20) & 1u);
        q[i] = k == kExpNan ? 0u : encode_value<TOP>(x[i], z, r);
    }
    store_codes<VEC>(codes, lane, len, q);
    if (lane == 0) *exps = (uint8_t)k;
}

template <bool VEC, typename PT, typename GT>
__device__ __forceinline__ void adamw8_block(const StepScalars& s, float keep, uint32_t key, PT* p,
                                             const GT* g, __nv_bfloat16* c, const StepArgs& a,
                                             int64_t sb, int lane, int len) {
    float pv[8], gv[8], mv[8], vv[8];
    const int64_t se = sb * kBlk;
    load<VEC>(g, lane, len, gv);
    load<VEC>(p, lane, len, pv);
    load_state<kTopM, VEC>(a.mc + se, a.mk[sb], lane, len, mv);
    load_state<kTopV, VEC>(a.vc + se, a.vk[sb], lane, len, vv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        adam_moments(s, gv[i], mv[i], vv[i]);
        pv[i] = adam_param(s, keep, pv[i], mv[i], vv[i]);
    }
    store<VEC>(p, lane, len, pv);
    if (c) store<VEC>(c, lane, len, pv);
    uint32_t am[8], av[8], w = 0;
    if constexpr (VEC) w = group_word(key, sb * 32 + lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = elem<VEC>(lane, i);
        if constexpr (!VEC) w = group_word(key, sb * 32 + (e >> 3));
        const uint32_t x = element_bits(w, e & 7);
        am[i] = (x >> 12) & 0xFFFF0u;
        av[i] = (x & 0xFFFFu) << 4;
    }
    store_state<kTopM, VEC, true>(a.mc + se, a.mk + sb, lane, len, mv, am);
    store_state<kTopV, VEC, true>(a.vc + se, a.vk + sb, lane, len, vv, av);
}

template <typename PT, typename GT, int N>
__global__ void __launch_bounds__(kThreads, 4)
k_adamw8(const __grid_constant__ TensorTable<N> t, const StepArgs a) {
    const StepScalars s = step_scalars(a);
    const int lane = threadIdx.x & 31;
    if (!s.skip) {
        const uint32_t key = step_key(a.seed, a.ctl->t + 1);
        uint32_t b = blockIdx.x * kWarps + (threadIdx.x >> 5);
        const uint32_t hop = gridDim.x * kWarps;
        int i = tensor_of(t, b);
        float keep = 0.0f;
        int known = -1;
        for (; b < t.nblk; b += hop) {
            while (b >= t.first[i + 1]) ++i;
            if (i != known) {
                keep = (float)(1.0 - s.lr * t.wd[i]);
                known = i;
            }
            const int64_t e = (int64_t)(b - t.first[i]) * kBlk, sb = t.blk0 + b;
            const int len = b + 1 == t.first[i + 1] ? t.last[i] & 0x1ff : kBlk;
            PT* p = static_cast<PT*>(t.p[i]) + e;
            const GT* g = static_cast<const GT*>(t.g[i]) + e;
            __nv_bfloat16* c = static_cast<__nv_bfloat16*>(t.c[i]);
            if (c) c += e;
            if (len == kBlk && (t.last[i] & kTabVec))
                adamw8_block<true>(s, keep, key, p, g, c, a, sb, lane, len);
            else
                adamw8_block<false>(s, keep, key, p, g, c, a, sb, lane, len);
        }
    }
    step_done(a, s.skip);
}

// The 8-bit states as values, and back (rounded to nearest even): one warp per block.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
k_adamw8_get(const uint8_t* mc, const uint8_t* vc, const uint8_t* mk, const uint8_t* vk,
             int64_t nblk, T* m, T* v) {
    const int lane = threadIdx.x & 31;
    const int64_t hop = (int64_t)gridDim.x * kWarps;
    for (int64_t b = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); b < nblk; b += hop) {
        float x[8];
        if (m) {
            load_state<kTopM, true>(mc + b * kBlk, mk[b], lane, kBlk, x);
            store<true>(m + b * kBlk, lane, kBlk, x);
        }
        if (v) {
            load_state<kTopV, true>(vc + b * kBlk, vk[b], lane, kBlk, x);
            store<true>(v + b * kBlk, lane, kBlk, x);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 4)
k_adamw8_set(uint8_t* mc, uint8_t* vc, uint8_t* mk, uint8_t* vk, int64_t nblk, const float* m,
             const float* v) {
    const int lane = threadIdx.x & 31;
    const int64_t hop = (int64_t)gridDim.x * kWarps;
    const uint32_t none[8] = {};
    for (int64_t b = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); b < nblk; b += hop) {
        float x[8];
        if (m) {
            load<true>(m + b * kBlk, lane, kBlk, x);
            store_state<kTopM, true, false>(mc + b * kBlk, mk + b, lane, kBlk, x, none);
        }
        if (v) {
            load<true>(v + b * kBlk, lane, kBlk, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] <= 0.0f ? 0.0f : x[i];
            store_state<kTopV, true, false>(vc + b * kBlk, vk + b, lane, kBlk, x, none);
        }
    }
}

// ------------------------------------------------------------------------------------------
// Global gradient norm: fp64 sums of squares in a fixed order (lane, warp, block, then the
// blocks' partial sums by the block that finishes last), so the result does not depend on which
// block that is.

constexpr int kNormBlocks = 148 * 8;

struct NormWork {              // ONEBIT_GRAD_NORM_BYTES; zero before the first call
    double sumsq;
    float norm, scale;
    uint32_t ticket;
    uint32_t pad[11];
    double part[kNormBlocks];
};

struct NormArgs {
    double max_norm;
    int32_t accumulate;   // add to work->sumsq instead of starting anew
    NormWork* work;
};

template <bool VEC, typename GT>
__device__ __forceinline__ double block_sumsq(const GT* g, int lane, int len, double acc) {
    float x[8];
    load<VEC>(g, lane, len, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = __fma_rn((double)x[i], (double)x[i], acc);
    return acc;
}

template <typename GT, int N>
__global__ void __launch_bounds__(kThreads, 8)
k_grad_norm(const __grid_constant__ TensorTable<N> t, const NormArgs a) {
    __shared__ double red[kWarps];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t b = blockIdx.x * kWarps + warp;
    const uint32_t hop = gridDim.x * kWarps;
    int i = tensor_of(t, b);
    double acc = 0.0;
    for (; b < t.nblk; b += hop) {
        while (b >= t.first[i + 1]) ++i;
        const int len = b + 1 == t.first[i + 1] ? t.last[i] & 0x1ff : kBlk;
        const GT* g = static_cast<const GT*>(t.g[i]) + (int64_t)(b - t.first[i]) * kBlk;
        if (len == kBlk && (t.last[i] & kTabVec))
            acc = block_sumsq<true>(g, lane, len, acc);
        else
            acc = block_sumsq<false>(g, lane, len, acc);
    }
    acc = warp_sum(acc);
    if (lane == 0) red[warp] = acc;
    __syncthreads();
    NormWork* w = a.work;
    if (threadIdx.x == 0) {
        w->part[blockIdx.x] = block_total(red);
        __threadfence();
        last = atomicAdd(&w->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double s = 0.0;
    for (uint32_t j = threadIdx.x; j < gridDim.x; j += kThreads) s += __ldcg(&w->part[j]);
    s = warp_sum(s);
    if (lane == 0) red[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        w->ticket = 0;
        const double sumsq = (a.accumulate ? w->sumsq : 0.0) + block_total(red);
        const double norm = sqrt(sumsq);
        w->sumsq = sumsq;
        w->norm = (float)norm;
        // a norm that is not finite gives a scale of NaN: the step that gets it is left out
        w->scale = !isfinite(w->norm) ? __int_as_float(0x7fffffff)
                   : norm > a.max_norm ? (float)(a.max_norm / norm) : 1.0f;
    }
}

}  // namespace onebit
