// adamw.cuh -- host side of the AdamW entry points (onebit_adamw_*, onebit_adamw8_*,
// onebit_grad_norm): argument checks and the launches. Included by onebit_adam.cu, whose error
// text and helpers it uses.
#pragma once

#include "adamw_clip.h"
#include "host.h"
#include "kernels_adamw.cuh"

static_assert(sizeof(StepCtl) == ONEBIT_ADAMW_CTL_BYTES, "control block");
static_assert(sizeof(NormWork) <= ONEBIT_GRAD_NORM_BYTES, "norm work");
static_assert(kBlk == ONEBIT_ADAMW_BLOCK, "state block");

namespace {

// Table sizes: a short one, so that small calls carry few parameters, and the largest that fits
// the 32,764 bytes a kernel's parameters may have; longer lists take several launches.
constexpr int kTabSmall = 64;
constexpr int kTabLarge = 800;

// The tensors of one call, as its kernels take them.
struct TensorList {
    int32_t n;
    const int64_t* numel;
    void* const* p;          // null: no parameters (grad norm)
    int32_t ptype;
    const void* const* g;
    int32_t gtype;
    void* const* c;          // null: no copies
    const double* wd;        // null: no decay
};

int check_list(const char* where, const TensorList& l, Ranges& ranges, int64_t* blocks) {
    if (l.n < 0) return bad(where, "negative number of tensors");
    if (l.n > 0 && (l.numel == nullptr || l.g == nullptr)) return bad(where, "null list");
    if (!known_dtype(l.gtype) || !known_dtype(l.ptype)) return bad(where, "unknown type");
    if (l.c != nullptr && l.ptype != ONEBIT_F32)
        return bad(where, "copies need float32 parameters");
    int64_t total = 0;
    for (int32_t i = 0; i < l.n; ++i) {
        const int64_t n = l.numel[i];
        if (n < 0 || n > ((int64_t)1 << 39)) return bad(where, "bad size of a tensor");
        if (n == 0) continue;
        total += ceil_div(n, kBlk);
        if (total > ((int64_t)1 << 40)) return bad(where, "too many elements");
        if (l.g[i] == nullptr || (l.p != nullptr && l.p[i] == nullptr) ||
            (l.c != nullptr && l.c[i] == nullptr))
            return bad(where, "null tensor");
        if (!aligned_to(l.g[i], width(l.gtype)) ||
            (l.p != nullptr && !aligned_to(l.p[i], width(l.ptype))) ||
            (l.c != nullptr && !aligned_to(l.c[i], 2)))
            return bad(where, "tensor not aligned to its elements", ONEBIT_ERR_ALIGN);
        if (l.wd != nullptr && !(std::isfinite(l.wd[i]) && l.wd[i] >= 0.0))
            return bad(where, "weight decay must be finite and >= 0");
    }
    const auto run = [&](int k, void* const* list, int64_t bytes, bool write) {
        if (list == nullptr) return;
        ranges.reserve(k, l.n);
        for (int32_t i = 0; i < l.n; ++i) ranges.add(k, list[i], l.numel[i] * bytes, write);
    };
    run(1, l.p, width(l.ptype), true);
    run(2, const_cast<void* const*>(l.g), width(l.gtype), false);
    run(3, l.c, 2, true);
    *blocks = total;
    return ONEBIT_OK;
}

// Tensors from `i` on into one table; returns the next one, the table being full or its block
// numbers near 32 bits.
template <int N>
int32_t fill(const TensorList& l, int32_t i, int64_t blk0, TensorTable<N>& t) {
    t.n = 0;
    t.blk0 = blk0;
    uint64_t b = 0;
    for (; i < l.n && t.n < N; ++i) {
        const int64_t n = l.numel[i];
        if (n == 0) continue;
        // the norm (no parameters) counts blocks from the vector that the tensor begins in
        const int64_t w = width(l.gtype);
        const int64_t lead =
            l.p == nullptr ? (int64_t)(reinterpret_cast<uintptr_t>(l.g[i]) % (8 * w)) / w : 0;
        const uint64_t nb = (uint64_t)ceil_div(n + lead, kBlk);
        if (t.n > 0 && b + nb > 0x80000000ull) break;
        const int k = t.n++;
        t.first[k] = (uint32_t)b;
        t.g[k] = static_cast<const char*>(l.g[i]) - lead * w;
        t.p[k] = l.p != nullptr ? l.p[i] : nullptr;
        t.c[k] = l.c != nullptr ? l.c[i] : nullptr;
        t.wd[k] = l.wd != nullptr ? l.wd[i] : 0.0;
        t.last[k] = (uint16_t)((n + lead - (int64_t)(nb - 1) * kBlk) | lead << kTabShift);
        if (aligned_to(t.g[k], 8 * width(l.gtype)) && aligned_to(t.p[k], 8 * width(l.ptype)) &&
            aligned16(t.c[k]))
            t.last[k] |= kTabVec;
        b += nb;
    }
    while (i < l.n && l.numel[i] == 0) ++i;  // empty ones at the end need no launch
    t.first[t.n] = (uint32_t)b;
    t.nblk = (uint32_t)b;
    return i;
}

unsigned grid_for(uint32_t nblk, int per_sm) {
    return (unsigned)std::min<int64_t>(std::max<int64_t>(ceil_div(nblk, kWarps), 1),
                                       kSms * per_sm);
}

// Queue `launch(table, last)` over the whole list, once at least.
template <int N, typename F>
int for_tables(const TensorList& l, F&& launch) {
    TensorTable<N> t;
    int32_t i = 0;
    int64_t blk0 = 0;
    do {
        i = fill(l, i, blk0, t);
        launch(t, i >= l.n);
        ONEBIT_CUDA(cudaGetLastError());
        blk0 += t.nblk;
    } while (i < l.n);
    return ONEBIT_OK;
}

// The table is up to 30 KB: it goes to the launch by address, not through a by-value stub.
template <int N, typename A>
void launch(void (*kernel)(TensorTable<N>, A), unsigned grid, const TensorTable<N>& t, const A& a,
            cudaStream_t st) {
    void* args[] = {const_cast<TensorTable<N>*>(&t), const_cast<A*>(&a)};
    (void)cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(kThreads), args,
                           0, st);
}

template <bool EIGHT, typename PT, typename GT, int N>
int queue_step(const TensorList& l, StepArgs a, cudaStream_t st) {
    return for_tables<N>(l, [&](const TensorTable<N>& t, bool last) {
        a.advance = last ? 1 : 0;
        if constexpr (EIGHT) {
            const uint32_t units = (uint32_t)ceil_div(t.nblk + (t.blk0 & (kUnit - 1)), kUnit);
            // fp32 parameters: shorter turns keep the streams closer together in memory (with bf16
            // gradients and copies, three times as many thread blocks as run at once against as
            // many: 128M parameters 352 us / 360, 32M 92.4 / 95.9, 16M 48.3 / 48.8; below that they
            // cost up to 5%, 5M 19.8 / 18.9, and up to 3M there are no more units than warps);
            // bf16 ones are bound by instructions (32M 68.2 / 64.7, 8M 23.4 / 21.4).
            const int per_sm = sizeof(PT) == 4 ? 3 * kStepBlocks : kStepBlocks;
            launch(k_adamw8<PT, GT, N>, grid_for(units, per_sm), t, a, st);
        } else {
            // fp32 parameters: two thread blocks per SM keep the eight streams closer together in
            // memory (all fp32, two against three: 333.6M parameters 1394 us / 1509, 32M 146 / 159,
            // 8M 41.0 / 43.4, 5M 27.7 / 28.5); calls that end after a few blocks a warp want three
            // (4M 23.1 / 23.1, 3M 18.9 / 18.3, 2M 14.7 / 13.7: equal at 16 blocks a warp, 4.85M).
            // bf16 ones need three for enough bytes in flight (333.6M 1274 / 1163, 8M 37.6 / 33.8).
            const int per_sm =
                sizeof(PT) == 4 && t.nblk >= (uint32_t)(kSms * kWarps * 16) ? 2 : kStepBlocks;
            launch(k_adamw<PT, GT, N>, grid_for(t.nblk, per_sm), t, a, st);
        }
    });
}

template <bool EIGHT, int N>
int queue_step(const TensorList& l, const StepArgs& a, cudaStream_t st) {
    const bool pf = l.ptype == ONEBIT_F32, gf = l.gtype == ONEBIT_F32;
    if (pf && gf) return queue_step<EIGHT, float, float, N>(l, a, st);
    if (pf) return queue_step<EIGHT, float, __nv_bfloat16, N>(l, a, st);
    if (gf) return queue_step<EIGHT, __nv_bfloat16, float, N>(l, a, st);
    return queue_step<EIGHT, __nv_bfloat16, __nv_bfloat16, N>(l, a, st);
}

int check_step(const char* where, StepArgs& a, double eps) {
    if (!std::isfinite(a.lr)) return bad(where, "lr must be finite");
    if (!(a.beta1 >= 0.0 && a.beta1 < 1.0) || !(a.beta2 >= 0.0 && a.beta2 < 1.0))
        return bad(where, "betas must lie in [0, 1)");
    if (!(std::isfinite(eps) && eps >= 0.0)) return bad(where, "eps must be finite and >= 0");
    if (a.bias != 0 && a.bias != 1) return bad(where, "bias_correction must be 0 or 1");
    if (a.ctl == nullptr) return bad(where, "null ctl");
    if (!aligned_to(a.ctl, 8) || !aligned_to(a.lr_dev, 8) || !aligned_to(a.scale, 4))
        return bad(where, "ctl, lr_dev or grad_scale not aligned", ONEBIT_ERR_ALIGN);
    const auto twice = [](float f) {
        uint32_t w;
        std::memcpy(&w, &f, 4);
        return (uint64_t)w << 32 | w;
    };
    a.eps = (float)eps;
    a.ombeta1 = 1.0 - a.beta1;
    a.ombeta2 = 1.0 - a.beta2;
    a.b1 = (float)a.beta1;
    a.omb1 = (float)a.ombeta1;
    a.b2 = (float)a.beta2;
    a.omb2 = (float)a.ombeta2;
    a.one2 = twice(1.0f);
    a.omb1_2 = twice(a.omb1);
    a.omb2_2 = twice(a.omb2);
    a.eps2 = twice(a.eps);
    // The fast 8-bit form takes square roots that flush below 2^-126, so a denominator may lose
    // up to 2^-63 / sqrt(c2), c2 >= 1 - beta2: below 2^-24 of eps if eps is at least this. Above
    // 2^60 a reciprocal could flush. Betas times a power of two have to be exact.
    a.fast = eps * std::sqrt(1.0 - a.beta2) >= 0x1p-39 && eps <= 0x1p60 &&
             (a.beta1 == 0.0 || a.beta1 >= 0x1p-64) && (a.beta2 == 0.0 || a.beta2 >= 0x1p-64);
    return ONEBIT_OK;
}

// The norm that comes before a clipped step.
struct Clip {
    double max_norm;
    void* work;
    bool* queued;  // set when the norm is on its way
};

int check_norm(const char* where, double max_norm, const void* work) {
    if (!(max_norm > 0.0)) return bad(where, "max_norm must be > 0");
    if (work == nullptr) return bad(where, "null work");
    if (!aligned_to(work, 8)) return bad(where, "work not aligned", ONEBIT_ERR_ALIGN);
    return ONEBIT_OK;
}

int queue_norm(const TensorList& l, const NormArgs& a, cudaStream_t st);

// Every check comes before anything is queued, the norm of a clipped step among it.
template <bool EIGHT>
int adamw_step(const char* where, const TensorList& l, StepArgs a, double eps, void* stream,
               Clip* clip = nullptr) {
    if (clip != nullptr) {
        const int rc = check_norm(where, clip->max_norm, clip->work);
        if (rc != ONEBIT_OK) return rc;
        a.scale = &static_cast<const NormWork*>(clip->work)->scale;
    }
    int rc = check_step(where, a, eps);
    if (rc != ONEBIT_OK) return rc;
    if (l.n > 0 && l.p == nullptr) return bad(where, "null list");
    Ranges ranges;
    int64_t blocks = 0;
    rc = check_list(where, l, ranges, &blocks);
    if (rc != ONEBIT_OK) return rc;
    if (blocks > 0) {
        if (EIGHT) {
            if (!a.mc || !a.vc || !a.mk || !a.vk) return bad(where, "null state");
            if (!aligned16(a.mc) || !aligned16(a.vc))
                return bad(where, "state not 16-byte aligned", ONEBIT_ERR_ALIGN);
            if (!aligned_to(a.mk, 4) || !aligned_to(a.vk, 4))
                return bad(where, "exponents not 4-byte aligned", ONEBIT_ERR_ALIGN);
            ranges.add(0, a.mc, blocks * kBlk, true);
            ranges.add(0, a.vc, blocks * kBlk, true);
            ranges.add(0, a.mk, blocks, true);
            ranges.add(0, a.vk, blocks, true);
        } else {
            if (!a.m || !a.v) return bad(where, "null state");
            if (!aligned_to(a.m, 32) || !aligned_to(a.v, 32))
                return bad(where, "state not 32-byte aligned", ONEBIT_ERR_ALIGN);
            ranges.add(0, a.m, blocks * kBlk * 4, true);
            ranges.add(0, a.v, blocks * kBlk * 4, true);
        }
    }
    ranges.add(0, a.ctl, sizeof(StepCtl), true);
    if (clip != nullptr)
        ranges.add(0, clip->work, ONEBIT_GRAD_NORM_BYTES, true);
    else
        ranges.add(0, a.scale, 4, false);
    ranges.add(0, a.lr_dev, 8, false);
    if (ranges.clash()) return bad(where, "tensors or states overlap");
    if (clip != nullptr) {
        *clip->queued = true;
        const TensorList g{l.n, l.numel, nullptr, ONEBIT_F32, l.g, l.gtype, nullptr, nullptr};
        rc = queue_norm(g, NormArgs{clip->max_norm, 0, static_cast<NormWork*>(clip->work)},
                        as_stream(stream));
        if (rc != ONEBIT_OK) return rc;
    }
    return l.n <= kTabSmall ? queue_step<EIGHT, kTabSmall>(l, a, as_stream(stream))
                            : queue_step<EIGHT, kTabLarge>(l, a, as_stream(stream));
}

StepArgs step_args(void* ctl, const float* grad_scale, const double* lr_dev, double lr,
                   double beta1, double beta2, int32_t bias) {
    StepArgs a{};
    a.lr = lr;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.lr_dev = lr_dev;
    a.scale = grad_scale;
    a.bias = bias;
    a.ctl = static_cast<StepCtl*>(ctl);
    return a;
}

int check_state8(const char* where, int64_t total, const void* mc, const void* vc,
                 const void* mk, const void* vk, const void* m, const void* v,
                 int64_t value_bytes) {
    if (total < 0 || total % kBlk != 0 || total > ((int64_t)1 << 46))
        return bad(where, "total must be a multiple of 256");
    if (total == 0) return ONEBIT_OK;
    if (m == nullptr && v == nullptr) return bad(where, "neither m nor v");
    if ((m != nullptr && (mc == nullptr || mk == nullptr)) ||
        (v != nullptr && (vc == nullptr || vk == nullptr)))
        return bad(where, "null state");
    if (!aligned16(mc) || !aligned16(vc))
        return bad(where, "state not 16-byte aligned", ONEBIT_ERR_ALIGN);
    if (!aligned_to(mk, 4) || !aligned_to(vk, 4))
        return bad(where, "exponents not 4-byte aligned", ONEBIT_ERR_ALIGN);
    if (!aligned_to(m, 8 * value_bytes) || !aligned_to(v, 8 * value_bytes))
        return bad(where, "values not aligned to eight of them", ONEBIT_ERR_ALIGN);
    return ONEBIT_OK;
}

// The converted vectors and the states they come from or go to: one writes, the other reads.
bool state8_clash(int64_t total, const void* mc, const void* vc, const void* mk, const void* vk,
                  const void* m, const void* v, int64_t value_bytes, bool to_state) {
    Ranges r;
    if (m != nullptr) {
        r.add(0, mc, total, to_state);
        r.add(0, mk, total / kBlk, to_state);
        r.add(0, m, total * value_bytes, !to_state);
    }
    if (v != nullptr) {
        r.add(0, vc, total, to_state);
        r.add(0, vk, total / kBlk, to_state);
        r.add(0, v, total * value_bytes, !to_state);
    }
    return r.clash();
}

template <typename GT, int N>
int queue_norm(const TensorList& l, NormArgs a, cudaStream_t st) {
    return for_tables<N>(l, [&](const TensorTable<N>& t, bool) {
        const uint32_t units = (uint32_t)ceil_div(t.nblk, kUnit);
        launch(k_grad_norm<GT, N>, grid_for(units, kNormPerSm), t, a, st);
        a.accumulate = 1;
    });
}

int queue_norm(const TensorList& l, const NormArgs& a, cudaStream_t st) {
    const bool small = l.n <= kTabSmall;
    if (l.gtype == ONEBIT_F32)
        return small ? queue_norm<float, kTabSmall>(l, a, st)
                     : queue_norm<float, kTabLarge>(l, a, st);
    return small ? queue_norm<__nv_bfloat16, kTabSmall>(l, a, st)
                 : queue_norm<__nv_bfloat16, kTabLarge>(l, a, st);
}

}  // namespace

extern "C" {

int onebit_adamw_layout(int32_t ntensors, const int64_t* numel, int64_t* offset, int64_t* total) {
    return guarded([&]() -> int {
        const char* where = "onebit_adamw_layout";
        if (ntensors < 0 || total == nullptr || (ntensors > 0 && (numel == nullptr || offset == nullptr)))
            return bad(where, "bad list");
        int64_t at = 0;
        for (int32_t i = 0; i < ntensors; ++i) {
            if (numel[i] < 0 || numel[i] > ((int64_t)1 << 39)) return bad(where, "bad size of a tensor");
            offset[i] = at;
            at += round_up(numel[i], kBlk);
            if (at > ((int64_t)1 << 48)) return bad(where, "too many elements");
        }
        *total = at;
        return ONEBIT_OK;
    });
}

int onebit_adamw_step(int32_t ntensors, const int64_t* numel, void* const* params,
                      int32_t param_dtype, const void* const* grads, int32_t grad_dtype,
                      void* const* copies, float* m, float* v, void* ctl,
                      const double* weight_decay, const float* grad_scale, const double* lr_dev,
                      double lr, double beta1, double beta2, double eps, int32_t bias_correction,
                      void* stream) {
    return guarded([&]() -> int {
        StepArgs a = step_args(ctl, grad_scale, lr_dev, lr, beta1, beta2, bias_correction);
        a.m = m;
        a.v = v;
        return adamw_step<false>("onebit_adamw_step",
                                 {ntensors, numel, params, param_dtype, grads, grad_dtype, copies,
                                  weight_decay},
                                 a, eps, stream);
    });
}

int onebit_adamw8_step(int32_t ntensors, const int64_t* numel, void* const* params,
                       int32_t param_dtype, const void* const* grads, int32_t grad_dtype,
                       void* const* copies, uint8_t* m, uint8_t* v, uint8_t* m_exp,
                       uint8_t* v_exp, void* ctl, uint64_t seed, const double* weight_decay,
                       const float* grad_scale, const double* lr_dev, double lr, double beta1,
                       double beta2, double eps, int32_t bias_correction, void* stream) {
    return guarded([&]() -> int {
        StepArgs a = step_args(ctl, grad_scale, lr_dev, lr, beta1, beta2, bias_correction);
        a.mc = m;
        a.vc = v;
        a.mk = m_exp;
        a.vk = v_exp;
        a.seed = seed;
        return adamw_step<true>("onebit_adamw8_step",
                                {ntensors, numel, params, param_dtype, grads, grad_dtype, copies,
                                 weight_decay},
                                a, eps, stream);
    });
}

int onebit_adamw8_get_state(int64_t total, const uint8_t* m, const uint8_t* v,
                            const uint8_t* m_exp, const uint8_t* v_exp, void* m_out, void* v_out,
                            int32_t out_dtype, void* stream) {
    return guarded([&]() -> int {
        const char* where = "onebit_adamw8_get_state";
        if (!known_dtype(out_dtype)) return bad(where, "unknown type");
        const int rc = check_state8(where, total, m, v, m_exp, v_exp, m_out, v_out, width(out_dtype));
        if (rc != ONEBIT_OK || total == 0) return rc;
        if (state8_clash(total, m, v, m_exp, v_exp, m_out, v_out, width(out_dtype), false))
            return bad(where, "values and states overlap");
        const int64_t nblk = total / kBlk;
        // a unit a warp, in the order in which the hardware takes them (333.6M parameters to fp32:
        // 496 us against 582 with two thread blocks per SM that walk over them)
        const unsigned grid =
            (unsigned)std::min<int64_t>(ceil_div(nblk, kWarps * kUnit), 1 << 30);
        if (out_dtype == ONEBIT_F32)
            k_adamw8_get<<<grid, kThreads, 0, as_stream(stream)>>>(
                m, v, m_exp, v_exp, nblk, static_cast<float*>(m_out), static_cast<float*>(v_out));
        else
            k_adamw8_get<<<grid, kThreads, 0, as_stream(stream)>>>(
                m, v, m_exp, v_exp, nblk, static_cast<__nv_bfloat16*>(m_out),
                static_cast<__nv_bfloat16*>(v_out));
        ONEBIT_CUDA(cudaGetLastError());
        return ONEBIT_OK;
    });
}

int onebit_adamw8_set_state(int64_t total, uint8_t* m, uint8_t* v, uint8_t* m_exp, uint8_t* v_exp,
                            const float* m_in, const float* v_in, void* stream) {
    return guarded([&]() -> int {
        const char* where = "onebit_adamw8_set_state";
        const int rc = check_state8(where, total, m, v, m_exp, v_exp, m_in, v_in, 4);
        if (rc != ONEBIT_OK || total == 0) return rc;
        if (state8_clash(total, m, v, m_exp, v_exp, m_in, v_in, 4, true))
            return bad(where, "values and states overlap");
        const int64_t nblk = total / kBlk;
        const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(nblk, kWarps * kUnit), kSms * 64);
        k_adamw8_set<<<grid, kThreads, 0, as_stream(stream)>>>(m, v, m_exp, v_exp, nblk, m_in, v_in);
        ONEBIT_CUDA(cudaGetLastError());
        return ONEBIT_OK;
    });
}

int onebit_grad_norm(int32_t ntensors, const int64_t* numel, const void* const* grads,
                     int32_t grad_dtype, double max_norm, int32_t accumulate, void* work,
                     void* stream) {
    return guarded([&]() -> int {
        const char* where = "onebit_grad_norm";
        if (accumulate != 0 && accumulate != 1) return bad(where, "accumulate must be 0 or 1");
        int rc = check_norm(where, max_norm, work);
        if (rc != ONEBIT_OK) return rc;
        const TensorList l{ntensors, numel, nullptr, ONEBIT_F32, grads, grad_dtype, nullptr, nullptr};
        Ranges ranges;
        int64_t blocks = 0;
        rc = check_list(where, l, ranges, &blocks);
        if (rc != ONEBIT_OK) return rc;
        ranges.add(0, work, ONEBIT_GRAD_NORM_BYTES, true);
        if (ranges.clash()) return bad(where, "work overlaps a gradient");
        return queue_norm(l, NormArgs{max_norm, accumulate, static_cast<NormWork*>(work)},
                          as_stream(stream));
    });
}

int onebit_internal_adamw_clipped_step(const OneBitAdamwClip* c, bool* queued) {
    return guarded([&]() -> int {
        StepArgs a = step_args(c->ctl, nullptr, c->lr_dev, c->lr, c->beta1, c->beta2,
                               c->bias_correction);
        const TensorList l{c->ntensors, c->numel, c->params, c->param_dtype, c->grads,
                           c->grad_dtype, c->copies, c->weight_decay};
        Clip clip{c->max_norm, c->work, queued};
        *queued = false;
        if (c->eight) {
            a.mc = static_cast<uint8_t*>(c->m);
            a.vc = static_cast<uint8_t*>(c->v);
            a.mk = c->m_exp;
            a.vk = c->v_exp;
            a.seed = c->seed;
            return adamw_step<true>("onebit_adamw8_step", l, a, c->eps, c->stream, &clip);
        }
        a.m = static_cast<float*>(c->m);
        a.v = static_cast<float*>(c->v);
        return adamw_step<false>("onebit_adamw_step", l, a, c->eps, c->stream, &clip);
    });
}

}  // extern "C"
