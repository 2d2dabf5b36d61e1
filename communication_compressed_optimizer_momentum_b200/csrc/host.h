// host.h -- what the host sides of the entry points share: the error text and the checks' helpers.
// Included by onebit_adam.cu alone.
#pragma once

#include <algorithm>
#include <cstdint>
#include <string>
#include <vector>

#include <cuda_runtime.h>

#include "onebit_adam.h"

namespace {

thread_local std::string g_last_error;  // of onebit_last_error

constexpr int kSms = 148;

int cuda_fail(cudaError_t e) {
    g_last_error = cudaGetErrorString(e);
    return ONEBIT_ERR_CUDA;
}

#define ONEBIT_CUDA(call)                                 \
    do {                                                  \
        cudaError_t e_ = (call);                          \
        if (e_ != cudaSuccess) return cuda_fail(e_);      \
    } while (0)

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// Half-open address ranges of one call: what it writes must not overlap anything else, or the
// result would depend on the order in which the blocks run. Ranges come in runs (a list of
// tensors each), which are nearly in ascending order in most programs: merges settle it, and
// nothing is sorted (a step over 800 separately allocated tensors: 49 us, against 55 sorted).
struct Ranges {
    struct R {
        uintptr_t lo, hi;
        bool write;
    };
    static constexpr int kRuns = 4;
    std::vector<R> r[kRuns];
    void reserve(int run, int32_t n) { r[run].reserve((size_t)std::max(n, 0)); }
    void add(int run, const void* p, int64_t bytes, bool write) {
        if (p != nullptr && bytes > 0) {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
            r[run].push_back({lo, lo + (uintptr_t)bytes, write});
        }
    }
    static bool by(const R& a, const R& b) { return a.lo < b.lo; }
    // Ascending order by merging what is in order already: allocators give addresses in few runs.
    static void order(std::vector<R>& v) {
        std::vector<size_t> cut{0};
        for (size_t i = 1; i < v.size(); ++i)
            if (by(v[i], v[i - 1])) cut.push_back(i);
        if (cut.size() > 16) return std::sort(v.begin(), v.end(), by);
        cut.push_back(v.size());
        while (cut.size() > 2) {
            std::vector<size_t> next;
            size_t k = 0;
            for (; k + 2 < cut.size(); k += 2) {
                std::inplace_merge(v.begin() + cut[k], v.begin() + cut[k + 1],
                                   v.begin() + cut[k + 2], by);
                next.push_back(cut[k]);
            }
            for (; k < cut.size(); ++k) next.push_back(cut[k]);
            cut.swap(next);
        }
    }
    bool clash() {
        const R *at[kRuns], *end[kRuns];
        int n = 0;
        for (auto& run : r) {
            if (run.empty()) continue;
            order(run);
            at[n] = run.data();
            end[n++] = run.data() + run.size();
        }
        uintptr_t any = 0, written = 0;
        while (n > 0) {
            int k = 0;
            for (int j = 1; j < n; ++j)
                if (at[j]->lo < at[k]->lo) k = j;
            const R& x = *at[k];
            if (x.lo < written || (x.write && x.lo < any)) return true;
            any = std::max(any, x.hi);
            if (x.write) written = std::max(written, x.hi);
            if (++at[k] == end[k]) {
                --n;
                at[k] = at[n];
                end[k] = end[n];
            }
        }
        return false;
    }
};

int bad(const char* where, const std::string& why, int code = ONEBIT_ERR_ARG) {
    g_last_error = std::string(where) + ": " + why;
    return code;
}

inline bool aligned_to(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline bool known_dtype(int32_t t) { return t == ONEBIT_F32 || t == ONEBIT_BF16; }
inline int64_t width(int32_t t) { return t == ONEBIT_F32 ? 4 : 2; }

// No C++ exception leaves a C entry point: the lists are the only thing that allocates. The reason
// is short enough to need no memory itself.
template <typename F>
int guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        g_last_error = "no host memory";
        return ONEBIT_ERR_SPACE;
    }
}

}  // namespace
