// tkq_flat.cuh -- the walk of a flat stream over the 128-channel groups of a
// row-major matrix (swiglu_flat.cu, swiglu_ckpt.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace tkq {

// One lane's place in the walk: unit u, its group g, the group's row t and
// block j (0 <= j < GH).  next() moves to unit u + step, i.e. group g + 4 step,
// with the row and block advanced by (dt, dj) = divmod(4 step, GH) and one
// carry.
struct Walk {
    int64_t u, g, t;
    int j;
    int64_t dt;
    int dj, GH;

    __device__ __forceinline__ Walk(int64_t u0, int sub, int64_t step, int gh) : GH(gh) {
        u = u0;
        g = u0 * 4 + sub;
        t = g / gh;
        j = static_cast<int>(g - t * gh);
        dt = (step * 4) / gh;
        dj = static_cast<int>(step * 4 - dt * gh);
    }
    __device__ __forceinline__ void next(int64_t step) {
        u += step;
        g += step * 4;
        t += dt;
        j += dj;
        if (j >= GH) {
            j -= GH;
            ++t;
        }
    }
};

}  // namespace tkq
