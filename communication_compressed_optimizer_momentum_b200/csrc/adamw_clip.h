// adamw_clip.h -- the clipped step as binding.cpp asks the library for it: the gradients' norm, then
// the step that takes its scale. Not part of the C ABI (a caller of that has the two entry points);
// one call, because all arguments of both have to be checked before the norm is queued, and to check
// the lists twice would cost the host as much again.
#pragma once

#include <cstdint>

struct OneBitAdamwClip {
    int32_t ntensors;
    const int64_t* numel;
    void* const* params;
    int32_t param_dtype;
    const void* const* grads;
    int32_t grad_dtype;
    void* const* copies;           // or null
    void *m, *v;                   // fp32 states, or with 8 bits codes ...
    uint8_t *m_exp, *v_exp;        // ... and exponents
    bool eight;
    uint64_t seed;
    void* ctl;
    const double* weight_decay;    // or null
    double max_norm;
    void* work;                    // of onebit_grad_norm; its scale is the step's grad_scale
    const double* lr_dev;          // or null
    double lr, beta1, beta2, eps;
    int32_t bias_correction;
    void* stream;
};

// A status of onebit_status. queued: whether any of the work has been queued.
extern "C" int onebit_internal_adamw_clipped_step(const OneBitAdamwClip* c, bool* queued);
