// The pyramid's node mean, shared by every kernel that forms nodes (so that all of them agree bit for
// bit).
#pragma once

#include <stdint.h>

namespace pisa {

// Mean of the children of node c (in the level below, whose row j sits at rows[(j - first) *
// stride]) weighted by the level-0 blocks holding keys that each child covers; 4 floats at the
// caller's column offset. n0: level-0 blocks that hold keys; width_below: f^(l-1).
__device__ __forceinline__ float4 node_mean4(const float* rows, int64_t first, int stride, int64_t c, int factor,
                                             int64_t n_below, int64_t width_below, int64_t n0) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    int64_t wsum = 0;
    for (int u = 0; u < factor; ++u) {
        const int64_t ch = c * factor + u;
        if (ch >= n_below) break;
        const int64_t lo = ch * width_below;
        const int64_t hi = min((ch + 1) * width_below, n0);
        if (hi <= lo) break;  // this child and the ones after it hold no key
        const float w = static_cast<float>(hi - lo);
        const float4 v = *reinterpret_cast<const float4*>(rows + (ch - first) * stride);
        acc.x = __fmaf_rn(w, v.x, acc.x);
        acc.y = __fmaf_rn(w, v.y, acc.y);
        acc.z = __fmaf_rn(w, v.z, acc.z);
        acc.w = __fmaf_rn(w, v.w, acc.w);
        wsum += hi - lo;
    }
    const float inv = wsum > 0 ? 1.0f / static_cast<float>(wsum) : 0.f;
    return make_float4(__fmul_rn(acc.x, inv), __fmul_rn(acc.y, inv), __fmul_rn(acc.z, inv), __fmul_rn(acc.w, inv));
}

}  // namespace pisa
