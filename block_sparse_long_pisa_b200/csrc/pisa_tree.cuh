// What the two kernels of the tree attention share: the cut of the work into runs, and small helpers.
#pragma once

#include <stdint.h>

#include "pisa_device.cuh"

namespace pisa {

constexpr uint32_t kTreeDetail = kKernTree << 8;
constexpr int kTreeUMin = -100;  // smallest unit exponent of O (e4m3)

// ---------------------------------------------------------------- the runs

// Units of one row tile of sequence b: the cache's, then one for the drafted tokens.
__device__ __forceinline__ int tree_len(const TreeParams& p, int b) {
    return min(max(p.len[b], 0), p.cap);
}
__device__ __forceinline__ int tree_units(const TreeParams& p, int len) {
    return p.topk > 0 ? 1 + p.topk * p.upb + (max(len - p.seq, 0) + 63) / 64 : 1 + (len + 63) / 64;
}

// The whole job and one position in it, formed by one warp.
struct TreeJob {
    int64_t total;   // units of all row tiles
    int64_t runs;    // runs that hold any (equal to the grid unless there are fewer units)
    __device__ __forceinline__ int64_t begin(int64_t c) const { return total * c / runs; }
    // run that holds unit x
    __device__ __forceinline__ int64_t run_of(int64_t x) const {
        int64_t c = x * runs / total;
        while (c + 1 < runs && begin(c + 1) <= x) ++c;
        while (begin(c) > x) --c;
        return c;
    }
};

__device__ __forceinline__ TreeJob tree_job(const TreeParams& p) {
    const int lane = threadIdx.x & 31;
    int64_t sum = 0;
    for (int b = lane; b < p.B; b += 32) sum += tree_units(p, tree_len(p, b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    TreeJob j;
    j.total = sum * p.rows_per_seq;
    j.runs = min(static_cast<int64_t>(p.runs), (j.total + p.min_units - 1) / p.min_units);
    return j;
}

// Row tile and unit at position x (whole warp).
__device__ __forceinline__ void tree_find(const TreeParams& p, int64_t x, int64_t& tile, int& unit) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int u = b < p.B ? tree_units(p, tree_len(p, b)) : 0;
        const int64_t mine = static_cast<int64_t>(u) * p.rows_per_seq;
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += y;
        }
        upto += before;
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, b < p.B && x < upto);
        if (hit != 0) {
            const int l = __ffs(hit) - 1;
            const int64_t start = __shfl_sync(0xFFFFFFFFu, upto - mine, l);
            const int ul = __shfl_sync(0xFFFFFFFFu, u, l);
            const int64_t rel = x - start;
            tile = static_cast<int64_t>(b0 + l) * p.rows_per_seq + rel / ul;
            unit = static_cast<int>(rel % ul);
            return;
        }
        before = __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    tile = static_cast<int64_t>(p.B) * p.rows_per_seq;
    unit = 0;
}

__device__ __forceinline__ float pow2i(int e) {  // e in [-126, 127]
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace pisa
