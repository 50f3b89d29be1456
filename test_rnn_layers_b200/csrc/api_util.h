// api_util.h -- what the C-ABI layers share: the thread's last-error message and the argument checks.
// Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ttt.h"

namespace ttt {

// Set this thread's last-error message and return `code`; clear it and return TTT_OK.
int fail(int code, const char* fmt, ...);
int ok();

inline int cuda_fail(cudaError_t e, const char* what) {
    return fail(TTT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// A byte range [p, p + n) of one argument, for the overlap checks.
struct Span {
    const char* name;
    const void* p;
    size_t n;
};

inline bool overlaps(const Span& x, const Span& y) {
    if (!x.p || !y.p || x.n == 0 || y.n == 0) return false;
    auto a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return a < b + y.n && b < a + x.n;
}

// outputs must not overlap inputs or each other; `same_ok` lists (output, input) index pairs
// allowed to be the SAME buffer (identical pointer and size: an in-place state update).
inline int check_aliasing(const Span* in, int nin, const Span* out, int nout,
                   const int (*same_ok)[2] = nullptr, int nsame = 0) {
    for (int o = 0; o < nout; ++o) {
        for (int i = 0; i < nin; ++i) {
            if (!overlaps(out[o], in[i])) continue;
            bool allowed = false;
            for (int k = 0; k < nsame; ++k)
                if (same_ok[k][0] == o && same_ok[k][1] == i && out[o].p == in[i].p && out[o].n == in[i].n)
                    allowed = true;
            if (!allowed)
                return fail(TTT_ERR_ALIAS, "output %s overlaps input %s", out[o].name, in[i].name);
        }
        for (int p = o + 1; p < nout; ++p)
            if (overlaps(out[o], out[p]))
                return fail(TTT_ERR_ALIAS, "outputs %s and %s overlap", out[o].name, out[p].name);
    }
    return TTT_OK;
}

}  // namespace ttt
