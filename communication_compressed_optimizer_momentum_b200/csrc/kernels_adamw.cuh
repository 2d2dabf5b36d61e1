// kernels_adamw.cuh -- AdamW over a list of tensors for B200 (sm_100a): the step with 32-bit and
// with 8-bit states, the global gradient norm, and the conversion of the 8-bit states.
//
// Work unit: a BLOCK of kBlk = 256 consecutive elements of one tensor, owned by one warp, eight
// elements a lane. The states of all tensors lie in one flat vector in which every tensor begins
// at a block boundary, so a block of a tensor is a block of the state. The tensors' addresses
// travel in the kernel parameters (TensorTable, up to 30 KB), so a call queues one launch for up to
// 800 tensors and keeps nothing: no table in device memory to upload, to go stale, or to be shared.
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
constexpr int kStepBlocks = 3;        // thread blocks per SM of the steps: 80 registers a thread
constexpr int kUnit = 4;              // blocks that a warp of the 8-bit step takes at a time
constexpr uint32_t kGolden = 0x9E3779B9u;
// TensorTable::last: elements in the last block (9 bits), elements of the first block that lie
// before the tensor (3 bits; the norm's blocks begin at addresses that take ld8), and whether all
// addresses take ld8 and st8.
constexpr int kTabShift = 9;
constexpr uint16_t kTabVec = 0x8000u;

// The tensors of one launch (empty ones left out).
template <int N>
struct TensorTable {
    int32_t n;
    uint32_t nblk;           // blocks of all tensors
    int64_t blk0;            // state block of the first
    uint32_t first[N + 1];   // first block of each tensor, counted from blk0
    uint16_t last[N];        // see kTabShift, kTabVec
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
    double lr, beta1, beta2, ombeta1, ombeta2;
    const double* lr_dev;    // overrides lr (or null)
    const float* scale;      // factor on every gradient (or null)
    float eps;
    int32_t bias;            // bias correction on
    int32_t advance;         // this launch is the step's last: count it
    float b1, omb1, b2, omb2;  // beta1, 1 - beta1, beta2, 1 - beta2
    uint64_t one2, omb1_2, omb2_2, eps2;  // 1, 1 - beta1, 1 - beta2, eps, each twice as fp32
    uint64_t seed;           // 8-bit states: stochastic rounding
    int32_t fast;            // eps allows the approximations
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
//
// fp32 as one 32-byte access: two 16-byte ones would each touch every other half of the warp's
// sectors, which moves the stores twice (the step on 333.6M fp32 parameters: 1557 us against 1707).

__device__ __forceinline__ void ld8(const float* p, float (&o)[8]) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]),
                   "=f"(o[6]), "=f"(o[7])
                 : "l"(p));
}

__device__ __forceinline__ void st8(float* p, const float (&o)[8]) {
    asm volatile("st.global.v8.f32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(o[0]), "f"(o[1]),
                 "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7]), "l"(p)
                 : "memory");
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
// ld8), else every 32nd, so that a warp's accesses are contiguous at any alignment.
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

// This warp within its thread block, in a form that lets the compiler keep what follows from it
// in uniform registers (8-bit step, fp32 and bf16: 787 -> 729 us, all bf16 648 -> 623).
__device__ __forceinline__ uint32_t warp_of_block() {
    return __shfl_sync(kFull, threadIdx.x >> 5, 0);
}

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

// Elements of tensor i's first block that lie before it.
template <int N>
__device__ __forceinline__ int lead_in(const TensorTable<N>& t, int i) {
    return (t.last[i] >> kTabShift) & 7;
}

// A warp's turn: kUnit blocks that begin at a multiple of it (`lead`: blocks before the launch's
// first within its unit), or what there is of them. i: the tensor of the first, carried along.
template <int N>
struct Unit {
    uint32_t b, n;  // first block (counted from blk0), number of blocks
    bool whole;     // kUnit whole blocks of tensor i, aligned
    __device__ __forceinline__ Unit(const TensorTable<N>& t, uint32_t lead, uint32_t u, int& i) {
        b = u * kUnit > lead ? u * kUnit - lead : 0u;
        n = min((u + 1) * kUnit - lead, t.nblk) - b;
        while (b >= t.first[i + 1]) ++i;
        const uint32_t full = t.first[i + 1] - ((t.last[i] & 0x1ff) == kBlk ? 0u : 1u);
        whole = n == kUnit && b + n <= full && (t.last[i] & kTabVec) &&
                b >= t.first[i] + (lead_in(t, i) ? 1u : 0u);
    }
};
template <int N>
__device__ __forceinline__ uint32_t units_of(const TensorTable<N>& t, uint32_t lead) {
    return t.nblk > 0 ? (t.nblk + lead + kUnit - 1) / kUnit : 0u;
}
template <int N>
__device__ __forceinline__ int first_tensor(const TensorTable<N>& t, uint32_t lead, uint32_t u) {
    return tensor_of(t, u * kUnit > lead ? u * kUnit - lead : 0u);
}

// The step's scalars that depend on device values: fp64, rounded once.
struct StepScalars {
    float step, r2, scale;
};

__device__ __forceinline__ double mean_of_ones(double c, double beta, double omb) {
    return __dadd_rn(__dmul_rn(beta, c), omb);
}

__device__ __forceinline__ double step_lr(const StepArgs& a) { return a.lr_dev ? *a.lr_dev : a.lr; }

__device__ __forceinline__ StepScalars step_scalars(const StepArgs& a) {
    StepScalars s;
    s.scale = a.scale ? *a.scale : 1.0f;
    double c1 = 1.0, c2 = 1.0;
    if (a.bias) {
        c1 = mean_of_ones(a.ctl->c1, a.beta1, a.ombeta1);
        c2 = mean_of_ones(a.ctl->c2, a.beta2, a.ombeta2);
    }
    s.step = (float)(step_lr(a) / c1);
    s.r2 = (float)(1.0 / sqrt(c2));
    return s;
}

// What a tensor's parameters are multiplied by: 1 - lr wd.
__device__ __forceinline__ float keep_of(const StepArgs& a, double wd) {
    return (float)__dsub_rn(1.0, __dmul_rn(step_lr(a), wd));
}

// Count the step once every block of its last launch is done. Only reads of ctl have to come
// before this, and every thread has used what it read by the barrier: no fence (which small calls
// feel: 240 tensors of 1 to 4 thousand elements take 6.2 us with one, 5.7 without).
__device__ __forceinline__ void step_done(const StepArgs& a, bool skip) {
    if (!a.advance) return;
    __syncthreads();
    if (threadIdx.x != 0) return;
    StepCtl* c = a.ctl;
    if (atomicAdd(&c->ticket, 1u) != gridDim.x - 1) return;
    c->ticket = 0;
    if (skip) {
        c->skipped += 1;
    } else {
        c->t += 1;
        c->c1 = mean_of_ones(c->c1, a.beta1, a.ombeta1);
        c->c2 = mean_of_ones(c->c2, a.beta2, a.ombeta2);
    }
}

//   m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2
__device__ __forceinline__ void adam_moments(const StepScalars& s, const StepArgs& a, float g,
                                             float& m, float& v) {
    const float gs = __fmul_rn(g, s.scale);
    m = __fadd_rn(__fmul_rn(a.b1, m), __fmul_rn(a.omb1, gs));
    v = __fadd_rn(__fmul_rn(a.b2, v), __fmul_rn(a.omb2, __fmul_rn(gs, gs)));
}

//   p = p (1 - lr wd) - (lr / c1) * m / (sqrt(v) / sqrt(c2) + eps)
__device__ __forceinline__ float adam_param(const StepScalars& s, const StepArgs& a, float keep,
                                            float p, float m, float v) {
    const float den = __fadd_rn(__fmul_rn(__fsqrt_rn(v), s.r2), a.eps);
    return __fsub_rn(__fmul_rn(p, keep), __fmul_rn(s.step, __fdiv_rn(m, den)));
}

// ------------------------------------------------------------------------------------------
// 32-bit states

template <bool VEC, typename PT, typename GT>
__device__ __forceinline__ void adamw_block(const StepScalars& s, const StepArgs& a, float keep,
                                            PT* p, const GT* g, __nv_bfloat16* c, float* m,
                                            float* v, int lane, int len) {
    float pv[8], gv[8], mv[8], vv[8];
    load<VEC>(g, lane, len, gv);
    load<VEC>(m, lane, len, mv);
    load<VEC>(v, lane, len, vv);
    load<VEC>(p, lane, len, pv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        adam_moments(s, a, gv[i], mv[i], vv[i]);
        pv[i] = adam_param(s, a, keep, pv[i], mv[i], vv[i]);
    }
    store<VEC>(m, lane, len, mv);
    store<VEC>(v, lane, len, vv);
    store<VEC>(p, lane, len, pv);
    if (c) store<VEC>(c, lane, len, pv);
}

// Bound by HBM: 28 bytes a parameter (fp32, bf16 gradients and copies) and 51 instructions, at 0.33
// issued a cycle. A block a warp at a time; the warps that run at once supply the loads in flight.
// 333.6M parameters, one B200: all fp32 1400 us (102% of the measured copy bandwidth), with bf16
// gradients and copies 1455 us (98%), all bf16 1145 us (98%), all bf16 at odd addresses, where
// elements are accessed one by one, 1350 us (83%).
template <typename PT, typename GT, int N>
__global__ void __launch_bounds__(kThreads, kStepBlocks)
k_adamw(const __grid_constant__ TensorTable<N> t, const StepArgs a) {
    const StepScalars s = step_scalars(a);
    const int lane = threadIdx.x & 31;
    const bool skip = !isfinite(s.scale);
    if (!skip) {
        uint32_t b = blockIdx.x * kWarps + (threadIdx.x >> 5);
        const uint32_t hop = gridDim.x * kWarps;
        int i = tensor_of(t, b);
        float keep = 0.0f;
        int known = -1;
        for (; b < t.nblk; b += hop) {
            while (b >= t.first[i + 1]) ++i;
            if (i != known) {
                keep = keep_of(a, t.wd[i]);
                known = i;
            }
            const int64_t e = (int64_t)(b - t.first[i]) * kBlk, se = (t.blk0 + b) * kBlk;
            const int len = b + 1 == t.first[i + 1] ? t.last[i] & 0x1ff : kBlk;
            PT* p = static_cast<PT*>(t.p[i]) + e;
            const GT* g = static_cast<const GT*>(t.g[i]) + e;
            __nv_bfloat16* c = static_cast<__nv_bfloat16*>(t.c[i]);
            if (c) c += e;
            if (len == kBlk && (t.last[i] & kTabVec))
                adamw_block<true>(s, a, keep, p, g, c, a.m + se, a.v + se, lane, len);
            else
                adamw_block<false>(s, a, keep, p, g, c, a.m + se, a.v + se, lane, len);
        }
    }
    step_done(a, skip);
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
// probability of the remainder keeps the mean of v (and m) that of the exact recurrence, but for
// what 16 random bits lose: 2^-17 of a spacing a rounding, v low by up to 2^-20 / (1 - beta2) of
// itself (0.1 % at 0.999). A
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

// 32 random bits from 32: two rounds of xor-shift and odd multiplication. Nothing but a test of the
// bits' means and correlations speaks for the multipliers.
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

// A block's state in the plain form, a lane's elements 32 apart: codes to values, and values to
// codes with 20 random bits each.
template <int TOP>
__device__ __forceinline__ void load_state(const uint8_t* codes, uint32_t k, int lane, int len,
                                           float (&x)[8]) {
    float f1, f2;
    decode_factors<TOP>(k, f1, f2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t c = i * 32 + lane < len ? codes[i * 32 + lane] : 0u;
        const uint32_t z = TOP == kTopM ? (c & 127u) << 20 | (c & 128u) << 24 : c << 20;
        x[i] = __fmul_rn(__fmul_rn(__uint_as_float(z), f1), f2);
    }
}

template <int TOP>
__device__ __forceinline__ void store_state(uint8_t* codes, uint8_t* exps, int lane, int len,
                                            const float (&x)[8], const uint32_t (&random)[8]) {
    uint32_t largest = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i * 32 + lane < len) largest = max(largest, __float_as_uint(x[i]) & 0x7fffffffu);
    const uint32_t k = block_exponent(__reduce_max_sync(kFull, largest));
    float f1, f2;
    encode_factors<TOP>(k, f1, f2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t z = __float_as_uint(__fmul_rn(__fmul_rn(fabsf(x[i]), f1), f2));
        uint32_t c = (z + random[i]) >> 20;
        c = TOP == kTopM ? c | ((__float_as_uint(x[i]) >> 24) & 128u)
                         : max(c, min(__float_as_uint(x[i]), 1u));
        if (i * 32 + lane < len) codes[i * 32 + lane] = (uint8_t)(k == kExpNan ? 0u : c);
    }
    if (lane == 0) *exps = (uint8_t)k;
}

// The parameters' update of the 8-bit step. With `fast` (see the host's rule for eps) square root
// and reciprocal are the hardware's approximations, 2^-23 each, with subnormals flushed, which eps
// covers: the quotient is good to 2^-21 of itself, far below the rounding of p that follows.
__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float adam_param8(const StepScalars& s, const StepArgs& a, float keep,
                                             float p, float m, float v) {
    if (!a.fast) return adam_param(s, a, keep, p, m, v);
    const float den = __fmaf_rn(sqrt_approx(v), s.r2, a.eps);
    return __fmaf_rn(-s.step, __fmul_rn(m, rcp_approx(den)), __fmul_rn(p, keep));
}

// One block in the plainest form: any alignment, any length, any exponent.
template <typename PT, typename GT>
__device__ __forceinline__ void adamw8_block(const StepScalars& s, float keep, uint32_t key, PT* p,
                                             const GT* g, __nv_bfloat16* c, const StepArgs& a,
                                             int64_t sb, int lane, int len) {
    float pv[8], gv[8], mv[8], vv[8];
    const int64_t se = sb * kBlk;
    load<false>(g, lane, len, gv);
    load<false>(p, lane, len, pv);
    load_state<kTopM>(a.mc + se, a.mk[sb], lane, len, mv);
    load_state<kTopV>(a.vc + se, a.vk[sb], lane, len, vv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        adam_moments(s, a, gv[i], mv[i], vv[i]);
        pv[i] = adam_param8(s, a, keep, pv[i], mv[i], vv[i]);
    }
    store<false>(p, lane, len, pv);
    if (c) store<false>(c, lane, len, pv);
    uint32_t am[8], av[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = i * 32 + lane;
        const uint32_t x = element_bits(group_word(key, sb * 32 + (e >> 3)), e & 7);
        am[i] = (x >> 12) & 0xFFFF0u;
        av[i] = (x & 0xFFFFu) << 4;
    }
    store_state<kTopM>(a.mc + se, a.mk + sb, lane, len, mv, am);
    store_state<kTopV>(a.vc + se, a.vk + sb, lane, len, vv, av);
}

// The same block with a third of the instructions (103 -> 43 an element), which is what the 8-bit
// step is short of: at 10 bytes an element HBM leaves an SM about 42 issue slots. Same results, bit
// for bit. What makes it short:
//  - pairs of fp32 operations in one instruction (f32x2);
//  - decoding costs no multiplication: beta * F is exact (F is a power of two), so beta * m is
//    (beta F) * z with z the code moved into an fp32 pattern. That needs block exponents whose F
//    and 1 / F are normal numbers and whose codes are fp32 numbers (up to 141 for m, 11 to 157
//    for v: m below 2^15, v below 2^31); others, and blocks whose new exponents pass these, take
//    the plain form;
//  - the quotient of adam_param8;
//  - the random bits are added so that a code ends in the top byte of a word, where four words
//    are packed by byte permutes; fp32's sign leaves by the same shift.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1,%2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
    asm("mov.b64 {%0,%1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// The largest magnitude of three, or NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t block_largest(const float (&x)[8]) {
    const float t = max3(max3(x[0], x[1], x[2]), x[6], x[7]), u = max3(x[3], x[4], x[5]);
    return __reduce_max_sync(kFull, __float_as_uint(max3(t, u, u)));
}
// The top bytes of four words.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Eight values of a lane as they are loaded, to be widened when they are used.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    float x[8];
    __device__ __forceinline__ void load(const float* p) { ld8(p, x); }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = x[i];
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(p));
    }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(w[i] << 16);
            o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

template <typename PT, typename GT>
struct Block8 {
    Raw8<GT> g;
    Raw8<PT> p;
    uint2 m, v;
    __device__ __forceinline__ void load(const PT* pp, const GT* gg, const uint8_t* mc,
                                         const uint8_t* vc, int lane) {
        g.load(gg + lane * kBlkLane);
        p.load(pp + lane * kBlkLane);
        asm volatile("ld.global.v2.b32 {%0,%1}, [%2];"
                     : "=r"(m.x), "=r"(m.y)
                     : "l"(mc + lane * kBlkLane));
        asm volatile("ld.global.v2.b32 {%0,%1}, [%2];"
                     : "=r"(v.x), "=r"(v.y)
                     : "l"(vc + lane * kBlkLane));
    }
};

constexpr uint32_t kFastM = 141u, kFastV = 157u, kFastVLow = 11u;

// False, with nothing stored, if the block needs the plain form. km, kv: its exponents, replaced.
// G: the lane's place in the state / 8; key holds the place's upper half. The parameters are stored
// as soon as they are known, which frees their registers for the codes.
template <typename PT, typename GT, typename Out>
__device__ __forceinline__ bool adamw8_fast(const Block8<PT, GT>& in, const StepScalars& s,
                                            const StepArgs& a, float keep, uint32_t key, uint32_t G, uint32_t& km,
                                            uint32_t& kv, const Out& out) {
    if (max(km + (kFastV - kFastM), kv) > kFastV) return false;
    if (kv < kFastVLow && __any_sync(kFull, (in.v.x | in.v.y) != 0u)) return false;
    float pv[8], gv[8], mv[8], vv[8];
    in.g.get(gv);
    {
        // one2 is 1, but not to the compiler, which else contracts these products and sums
        const float b1 = __fmul_rn(a.b1, pow2((int)km - kTopM));
        const float b2 = __fmul_rn(a.b2, pow2((int)max(kv, kFastVLow) - kTopV));
        const uint64_t B1 = pack2(b1, b1), B2 = pack2(b2, b2), S = pack2(s.scale, s.scale);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float zm[2], zv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t wm = i < 4 ? in.m.x : in.m.y, wv = i < 4 ? in.v.x : in.v.y;
                const int q = (i + j) & 3;
                // code to the top byte, then its sign stays and the rest moves to bits 26..20
                zm[j] = __int_as_float(((int32_t)(wm << (24 - 8 * q)) >> 4) & 0x87F00000);
                zv[j] = __uint_as_float((q < 3 ? wv << (20 - 8 * q) : wv >> 4) & 0x0FF00000u);
            }
            const uint64_t g2 = mul2(pack2(gv[i], gv[i + 1]), S);
            unpack2(fma2(mul2(B1, pack2(zm[0], zm[1])), a.one2, mul2(a.omb1_2, g2)), mv[i], mv[i + 1]);
            unpack2(fma2(mul2(B2, pack2(zv[0], zv[1])), a.one2, mul2(a.omb2_2, mul2(g2, g2))),
                    vv[i], vv[i + 1]);
        }
    }
    // new exponents: (pattern of the largest + 0xFFFFF) without its mantissa, see block_exponent
    const uint32_t em = (block_largest(mv) + 0xFFFFFu) & 0xFF800000u;
    const uint32_t ev = (block_largest(vv) + 0xFFFFFu) & 0xFF800000u;
    if (em > kFastM << 23 || ev > kFastV << 23) return false;
    km = em >> 23;
    kv = ev >> 23;
    in.p.get(pv);
    {
        const uint64_t R2 = pack2(s.r2, s.r2), K = pack2(keep, keep),
                       M = pack2(-s.step, -s.step);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float d0, d1;
            unpack2(fma2(pack2(sqrt_approx(vv[i]), sqrt_approx(vv[i + 1])), R2, a.eps2), d0, d1);
            const uint64_t q = mul2(pack2(mv[i], mv[i + 1]), pack2(rcp_approx(d0), rcp_approx(d1)));
            unpack2(fma2(M, q, mul2(pack2(pv[i], pv[i + 1]), K)), pv[i], pv[i + 1]);
        }
    }
    out.params(pv);
    const float fm = __uint_as_float(((127u + kTopM) << 23) - em);
    const float fv = __uint_as_float(((127u + kTopV) << 23) - ev);
    const uint64_t FM = pack2(fm, fm), FV = pack2(fv, fv);
    const uint32_t w = mix32(G + key);
    uint32_t ym[8], yv[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float zm[2], zv[2];
        unpack2(mul2(pack2(mv[i], mv[i + 1]), FM), zm[0], zm[1]);
        unpack2(mul2(pack2(vv[i], vv[i + 1]), FV), zv[0], zv[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t x = w + (uint32_t)(i + j + 1) * kGolden;
            x ^= x >> 15;
            x *= 0x8A8866C7u;
            // bits for m: x's upper half; for v: lower half ^ upper half; each shifted up by 8
            const uint32_t hi = __byte_perm(x, 0, 0x4324), lo = __byte_perm(x, 0, 0x4104);
            ym[i + j] = ((__float_as_uint(zm[j]) << 4) + hi) |
                        (__float_as_uint(mv[i + j]) & 0x80000000u);
            yv[i + j] = (__float_as_uint(zv[j]) << 4) + (hi ^ lo);
        }
    }
    uint32_t c0 = top_bytes(yv[0], yv[1], yv[2], yv[3]), c1 = top_bytes(yv[4], yv[5], yv[6], yv[7]);
    // where a word has a zero byte: codes of 0 that stand for positive values become 1
    if ((((c0 - 0x01010101u) & ~c0) | ((c1 - 0x01010101u) & ~c1)) & 0x80808080u) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (vv[i] > 0.0f) yv[i] = max(yv[i], 1u << 24);
        c0 = top_bytes(yv[0], yv[1], yv[2], yv[3]);
        c1 = top_bytes(yv[4], yv[5], yv[6], yv[7]);
    }
    out.codes(
        make_uint2(top_bytes(ym[0], ym[1], ym[2], ym[3]), top_bytes(ym[4], ym[5], ym[6], ym[7])),
        make_uint2(c0, c1));
    return true;
}

__device__ __forceinline__ uint2& lane_codes(uint8_t* codes, int lane) {
    return *reinterpret_cast<uint2*>(codes + lane * kBlkLane);
}

// Element places between a warp's contiguous accesses (every 32nd) and its lanes' eight
// consecutive ones, through 1 KB of shared memory.
__device__ __forceinline__ void stage_in(float* sm, const float (&x)[8], int lane, float (&o)[8]) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) sm[i * 32 + lane] = x[i];
    __syncwarp();
    ld4(sm + lane * 8, reinterpret_cast<float(&)[4]>(o[0]));
    ld4(sm + lane * 8 + 4, reinterpret_cast<float(&)[4]>(o[4]));
}

__device__ __forceinline__ uint32_t low_bytes(int n) {  // a mask of the n lowest bytes
    return n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}

// One block of any alignment and length by the fast form, or the plain one where that must be.
template <typename PT, typename GT>
__device__ __forceinline__ void adamw8_single(const StepScalars& s, float keep, uint32_t key, PT* p,
                                              const GT* g, __nv_bfloat16* c, const StepArgs& a,
                                              int64_t sb, int lane, int len, float* sm) {
    uint8_t *mc = a.mc + sb * kBlk, *vc = a.vc + sb * kBlk;
    uint32_t km = a.mk[sb], kv = a.vk[sb];
    const uint2 om = lane_codes(mc, lane), ov = lane_codes(vc, lane);
    // both are loaded before the first wait of the warp (all bf16 at odd addresses, 333.6M
    // parameters: 1048 -> 960 us, fp32 1167 -> 1118)
    float gv[8], pv[8];
    load<false>(g, lane, len, gv);
    load<false>(p, lane, len, pv);
    Block8<float, float> in;
    stage_in(sm, gv, lane, in.g.x);
    stage_in(sm, pv, lane, in.p.x);
    // the codes behind the tensor count as 0 and stay as they are
    const uint32_t k0 = low_bytes(len - lane * 8), k1 = low_bytes(len - lane * 8 - 4);
    in.m = make_uint2(om.x & k0, om.y & k1);
    in.v = make_uint2(ov.x & k0, ov.y & k1);
    const int64_t G = sb * 32 + lane;
    struct {
        PT* p;
        __nv_bfloat16* c;
        uint8_t *mc, *vc;
        float* sm;
        uint2 om, ov;
        uint32_t k0, k1;
        int lane, len;
        __device__ __forceinline__ void params(const float (&x)[8]) const {
            float y[8];
            __syncwarp();
            st4(sm + lane * 8, reinterpret_cast<const float(&)[4]>(x[0]));
            st4(sm + lane * 8 + 4, reinterpret_cast<const float(&)[4]>(x[4]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = sm[i * 32 + lane];
            store<false>(p, lane, len, y);
            if (c) store<false>(c, lane, len, y);
        }
        __device__ __forceinline__ void codes(uint2 m, uint2 v) const {
            lane_codes(mc, lane) = make_uint2((m.x & k0) | (om.x & ~k0), (m.y & k1) | (om.y & ~k1));
            lane_codes(vc, lane) = make_uint2((v.x & k0) | (ov.x & ~k0), (v.y & k1) | (ov.y & ~k1));
        }
    } const out{p, c, mc, vc, sm, om, ov, k0, k1, lane, len};
    if (a.fast && adamw8_fast(in, s, a, keep, key + (uint32_t)(G >> 32) * kGolden, (uint32_t)G, km,
                              kv, out)) {
        if (lane == 0) {
            a.mk[sb] = (uint8_t)km;
            a.vk[sb] = (uint8_t)kv;
        }
    } else {
        adamw8_block(s, keep, key, p, g, c, a, sb, lane, len);
    }
}

template <typename PT>
struct Out8 {
    PT* p;
    __nv_bfloat16* c;
    uint8_t *mc, *vc;
    __device__ __forceinline__ void params(const float (&x)[8]) const {
        st8(p, x);
        if (c) st8(c, x);
    }
    __device__ __forceinline__ void codes(uint2 m, uint2 v) const {
        *reinterpret_cast<uint2*>(mc) = m;
        *reinterpret_cast<uint2*>(vc) = v;
    }
};

// A warp takes units of kUnit blocks that begin at a multiple of it in the state, so that a unit's
// exponents are one word: read and written byte by byte they cost a tenth of the step (bf16,
// 333.6M parameters, transfers alone: 606 us against 545 without them). The next block but one is
// loaded while a block is computed, within the 80 registers that let three thread blocks share an
// SM. Blocks that a unit does not hold in full (tensors' ends) or that are not aligned go one by
// one. 333.6M parameters, one B200: all fp32 811 us (101% of the measured copy bandwidth), with
// bf16 gradients and copies 851 us (96%), all bf16 623-642 us (80-82%; 43 instructions an element
// at 0.67 issued a cycle take longer than the transfers), fp32 at odd addresses 1118 us (73%).
template <typename PT, typename GT, int N>
__global__ void __launch_bounds__(kThreads, kStepBlocks)
k_adamw8(const __grid_constant__ TensorTable<N> t, const StepArgs a) {
    __shared__ __align__(16) float stage[kWarps][kBlk];
    const StepScalars s = step_scalars(a);
    const int lane = threadIdx.x & 31;
    const bool skip = !isfinite(s.scale);
    if (!skip) {
        const uint32_t key = step_key(a.seed, a.ctl->t + 1);
        const uint32_t lead = (uint32_t)t.blk0 & (kUnit - 1);
        const uint32_t units = units_of(t, lead);
        uint32_t u = blockIdx.x * kWarps + warp_of_block();
        int i = first_tensor(t, lead, u), known = -1;
        float keep = 0.0f;
        for (; u < units; u += gridDim.x * kWarps) {
            const Unit<N> at(t, lead, u, i);
            // blocks that are left to go one by one, one bit each
            uint32_t left = (1u << at.n) - 1u;
            if (a.fast && at.whole) {
                if (i != known) {
                    keep = keep_of(a, t.wd[i]);
                    known = i;
                }
                const int64_t e = (int64_t)(at.b - t.first[i]) * kBlk, sb = t.blk0 + at.b;
                PT* p = static_cast<PT*>(t.p[i]) + e;
                const GT* g = static_cast<const GT*>(t.g[i]) + e;
                __nv_bfloat16* c = static_cast<__nv_bfloat16*>(t.c[i]);
                if (c) c += e;
                uint8_t *mc = a.mc + sb * kBlk, *vc = a.vc + sb * kBlk;
                uint32_t mk = *reinterpret_cast<const uint32_t*>(a.mk + sb);
                uint32_t vk = *reinterpret_cast<const uint32_t*>(a.vk + sb);
                const int64_t G = sb * 32 + lane;
                const uint32_t kh = key + (uint32_t)(G >> 32) * kGolden;
                left = 0u;
                Block8<PT, GT> in[2];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    in[q].load(p + q * kBlk, g + q * kBlk, mc + q * kBlk, vc + q * kBlk, lane);
#pragma unroll
                for (int q = 0; q < kUnit; ++q) {
                    uint32_t km = mk & 0xffu, kv = vk & 0xffu;
                    const int o = q * kBlk + lane * kBlkLane;
                    const Out8<PT> out{p + o, c ? c + o : c, mc + o, vc + o};
                    if (!adamw8_fast(in[q % 2], s, a, keep, kh, (uint32_t)G + q * 32, km, kv, out))
                        left |= 1u << q;
                    // the new exponent goes in at the top as the old one leaves below
                    mk = __byte_perm(mk, km, 0x4321);
                    vk = __byte_perm(vk, kv, 0x4321);
                    const int l = q + 2;
                    if (l < kUnit)
                        in[l % 2].load(p + l * kBlk, g + l * kBlk, mc + l * kBlk, vc + l * kBlk,
                                       lane);
                }
                if (lane == 0) {
                    *reinterpret_cast<uint32_t*>(a.mk + sb) = mk;
                    *reinterpret_cast<uint32_t*>(a.vk + sb) = vk;
                }
                __syncwarp();
            }
            for (int k = i; left; left &= left - 1u) {
                const uint32_t q = at.b + __ffs(left) - 1;
                while (q >= t.first[k + 1]) ++k;
                const int64_t e = (int64_t)(q - t.first[k]) * kBlk;
                __nv_bfloat16* c = static_cast<__nv_bfloat16*>(t.c[k]);
                adamw8_single(s, keep_of(a, t.wd[k]), key, static_cast<PT*>(t.p[k]) + e,
                              static_cast<const GT*>(t.g[k]) + e, c ? c + e : c, a, t.blk0 + q,
                              lane, q + 1 == t.first[k + 1] ? t.last[k] & 0x1ff : kBlk,
                              stage[threadIdx.x >> 5]);
            }
        }
    }
    step_done(a, skip);
}

// The 8-bit states as values, and back (rounded to nearest even): units of kUnit blocks as in the
// step; all of m's values before v's, so that a warp writes 4 KB at a time. 333.6M parameters: to
// fp32 496 us (103% of the measured copy bandwidth), to bf16 295 us (104%), from fp32 484 us (105%).
template <int TOP>
__device__ __forceinline__ void decode8(uint2 w, uint32_t k, float (&x)[8]) {
    float f1, f2;
    decode_factors<TOP>(k, f1, f2);
    const bool one = k <= (uint32_t)TOP + 127u;  // 2^(k-TOP) is a normal number: one factor
    if (one) f1 = pow2((int)k - TOP);
    const uint64_t F1 = pack2(f1, f1), F2 = pack2(f2, f2);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t v = i < 4 ? w.x : w.y;
        float z[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int q = (i + j) & 3;
            z[j] = TOP == kTopM
                       ? __int_as_float(((int32_t)(v << (24 - 8 * q)) >> 4) & 0x87F00000)
                       : __uint_as_float((q < 3 ? v << (20 - 8 * q) : v >> 4) & 0x0FF00000u);
        }
        uint64_t r = mul2(pack2(z[0], z[1]), F1);
        if (!one) r = mul2(r, F2);
        unpack2(r, x[i], x[i + 1]);
    }
}

// Codes of a lane's eight values and the block's exponent.
template <int TOP>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], uint32_t& k) {
    k = min((block_largest(x) + 0xFFFFFu) >> 23, kExpNan);
    float f1, f2;
    encode_factors<TOP>(k, f1, f2);
    const uint64_t F1 = pack2(f1, f1), F2 = pack2(f2, f2);
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float z[2];
        unpack2(mul2(mul2(pack2(x[i], x[i + 1]), F1), F2), z[0], z[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w = __float_as_uint(z[j]) & 0x7fffffffu;
            uint32_t c = (w + 0x7FFFFu + ((w >> 20) & 1u)) << 4;
            if (TOP == kTopM)
                c |= __float_as_uint(x[i + j]) & 0x80000000u;
            else
                c = x[i + j] > 0.0f ? max(c, 1u << 24) : c;
            y[i + j] = k == kExpNan ? 0u : c;
        }
    }
    return make_uint2(top_bytes(y[0], y[1], y[2], y[3]), top_bytes(y[4], y[5], y[6], y[7]));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
k_adamw8_get(const uint8_t* mc, const uint8_t* vc, const uint8_t* mk, const uint8_t* vk,
             int64_t nblk, T* m, T* v) {
    const int lane = threadIdx.x & 31;
    const int64_t hop = (int64_t)gridDim.x * kWarps * kUnit;
    for (int64_t b = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kUnit; b < nblk;
         b += hop) {
        uint2 cm[kUnit], cv[kUnit];
        uint32_t km = 0u, kv = 0u;
        const bool full = b + kUnit <= nblk;
#pragma unroll
        for (int q = 0; q < kUnit; ++q) {
            const bool in = b + q < nblk;
            const int64_t e = (b + q) * kBlk + lane * kBlkLane;
            cm[q] = in && m ? *reinterpret_cast<const uint2*>(mc + e) : make_uint2(0u, 0u);
            cv[q] = in && v ? *reinterpret_cast<const uint2*>(vc + e) : make_uint2(0u, 0u);
        }
        if (full) {
            if (m) km = *reinterpret_cast<const uint32_t*>(mk + b);
            if (v) kv = *reinterpret_cast<const uint32_t*>(vk + b);
        } else {
            for (int q = 0; b + q < nblk; ++q) {
                if (m) km |= (uint32_t)mk[b + q] << (8 * q);
                if (v) kv |= (uint32_t)vk[b + q] << (8 * q);
            }
        }
        float x[8];
#pragma unroll
        for (int q = 0; q < kUnit; ++q) {
            if (!m || b + q >= nblk) break;
            decode8<kTopM>(cm[q], (km >> (8 * q)) & 0xffu, x);
            st8(m + (b + q) * kBlk + lane * kBlkLane, x);
        }
#pragma unroll
        for (int q = 0; q < kUnit; ++q) {
            if (!v || b + q >= nblk) break;
            decode8<kTopV>(cv[q], (kv >> (8 * q)) & 0xffu, x);
            st8(v + (b + q) * kBlk + lane * kBlkLane, x);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 3)
k_adamw8_set(uint8_t* mc, uint8_t* vc, uint8_t* mk, uint8_t* vk, int64_t nblk, const float* m,
             const float* v) {
    const int lane = threadIdx.x & 31;
    const int64_t hop = (int64_t)gridDim.x * kWarps * kUnit;
    for (int64_t b = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kUnit; b < nblk;
         b += hop) {
        float xm[2][8], xv[2][8];
        auto load = [&](int q) {
            const int64_t e = (b + q) * kBlk + lane * kBlkLane;
            if (b + q < nblk && m) ld8(m + e, xm[q % 2]);
            if (b + q < nblk && v) ld8(v + e, xv[q % 2]);
        };
        load(0);
        uint32_t wm = 0u, wv = 0u;
#pragma unroll
        for (int q = 0; q < kUnit; ++q) {
            if (q + 1 < kUnit) load(q + 1);
            if (b + q >= nblk) break;
            const int64_t e = (b + q) * kBlk + lane * kBlkLane;
            uint32_t k;
            if (m) {
                *reinterpret_cast<uint2*>(mc + e) = encode8<kTopM>(xm[q % 2], k);
                wm |= k << (8 * q);
            }
            if (v) {
                float (&x)[8] = xv[q % 2];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] <= 0.0f ? 0.0f : x[i];
                *reinterpret_cast<uint2*>(vc + e) = encode8<kTopV>(x, k);
                wv |= k << (8 * q);
            }
        }
        // the unit's exponents by its first lanes; a unit at the end may be short
        if (lane < kUnit && b + lane < nblk) {
            if (m) mk[b + lane] = (uint8_t)(wm >> (8 * lane));
            if (v) vk[b + lane] = (uint8_t)(wv >> (8 * lane));
        }
    }
}

// ------------------------------------------------------------------------------------------
// Global gradient norm: fp64 sums of squares in a fixed order (lane, warp, block, then the
// blocks' partial sums by the block that finishes last), so the result does not depend on which
// block that is.

// Thread blocks per SM of the norm: what keeps enough bf16 in flight (665M elements: 216 us with 4,
// 202 with 6), at fp32's best (194 with 4 and 6, 204 with 5 and 7).
constexpr int kNormPerSm = 6;
constexpr int kNormBlocks = 148 * kNormPerSm;

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

template <typename T>
__device__ __forceinline__ double sumsq8(const T& raw, double acc) {
    float x[8];
    raw.get(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = __fma_rn((double)x[i], (double)x[i], acc);
    return acc;
}

// Units as in the 8-bit step: four loads in flight, and the walk over the tensors once for four
// blocks. Bound by HBM: bf16, 665M elements: 202 us, 101% of the measured copy bandwidth (block by
// block 270: the walk; a sustained loop at the power cap 230); fp32, 333.6M: 194 us, 105%. The
// blocks are counted from the address before a tensor that takes vector loads, so that views at odd
// addresses are read as fast (333.6M: bf16 119 us, fp32 195; element by element 254 and 316).
template <typename GT, int N>
__global__ void __launch_bounds__(kThreads, kNormPerSm)
k_grad_norm(const __grid_constant__ TensorTable<N> t, const NormArgs a) {
    __shared__ double red[kWarps];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t units = units_of(t, 0u);
    uint32_t u = blockIdx.x * kWarps + warp;
    int i = first_tensor(t, 0u, u);
    double acc = 0.0;
    for (; u < units; u += gridDim.x * kWarps) {
        const Unit<N> at(t, 0u, u, i);
        if (at.whole) {
            const GT* g = static_cast<const GT*>(t.g[i]) + (int64_t)(at.b - t.first[i]) * kBlk +
                          lane * kBlkLane;
            Raw8<GT> x[kUnit];
#pragma unroll
            for (int q = 0; q < kUnit; ++q) x[q].load(g + q * kBlk);
#pragma unroll
            for (int q = 0; q < kUnit; ++q) acc = sumsq8(x[q], acc);
        } else {
            int k = i;
            for (uint32_t b = at.b; b < at.b + at.n; ++b) {
                while (b >= t.first[k + 1]) ++k;
                const int lo = b == t.first[k] ? lead_in(t, k) : 0;
                const int len = b + 1 == t.first[k + 1] ? t.last[k] & 0x1ff : kBlk;
                const GT* g = static_cast<const GT*>(t.g[k]) + (int64_t)(b - t.first[k]) * kBlk;
                if (lo == 0 && len == kBlk) {
                    Raw8<GT> x;
                    x.load(g + lane * kBlkLane);
                    acc = sumsq8(x, acc);
                } else {
                    Raw8<float> x;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = j * 32 + lane;
                        x.x[j] = e >= lo && e < len ? ld1(g + e) : 0.0f;
                    }
                    acc = sumsq8(x, acc);
                }
            }
        }
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
