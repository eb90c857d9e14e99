// What the two kernels of the tree attention share: the cut of the work into runs, and small helpers.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "pisa_device.cuh"

namespace pisa {

constexpr uint32_t kTreeDetail = kKernTree << 8;
// The reference of a row without a finite score so far: below every score, so that the first one moves it, and finite, so
// that a score of minus infinity stays one. (A reference of 0 would round scores below -126 away that come later.)
constexpr float kTreeNone = -3.402823466e+38f;

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

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---------------------------------------------------------------- operands

// A matrix descriptor's start moved by `bytes`.
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t two) {
    const uint32_t h = e4m3x2_f16x2<false>(two);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// One lane of the whole warp, in a form that the compiler knows to be one lane.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
// Barrier `bar` over `count` threads (whole warps); true if `x` holds in any of them.
__device__ __forceinline__ bool vote_any(uint32_t bar, uint32_t count, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x)), "r"(bar), "r"(count)
        : "memory");
    return r != 0;
}

// ---------------------------------------------------------------- the tiles

constexpr int kTreeMaxSlots = 4;  // of the K ring and of the V ring
constexpr int kTreeMeta = 8;      // entries (tiles and piece ends) whose description is kept
enum : int { kTileEnd = 0, kTileCache = 1, kTileDraft = 2 };

// A place in a ring: slot, parity of its current use, and uses so far.
struct RingAt {
    int s = 0, n = 0;
    uint32_t par = 0;
    __device__ __forceinline__ void next(int slots) {
        ++n;
        if (++s == slots) {
            s = 0;
            par ^= 1u;
        }
    }
};

// The entries of a CTA's pieces in order: issue(kind, plane, len, a0, a1) for every tile (PAIRS: of 128 keys, two
// units, first keys a0 and a1, a1 = -1 for none; else of one unit, a1 = -1), for the drafted tokens, and for the end of
// each piece. Run by a whole warp; `reports`: this warp records bad lengths and indices. Stops when ok is cleared.
template <bool PAIRS, class Issue>
__device__ __forceinline__ void tree_entries(const TreeParams& p, int64_t pos, int64_t end, int64_t tile, int unit,
                                             bool reports, bool& ok, Issue issue) {
    const int lane = threadIdx.x & 31;
    while (pos < end && ok) {
        const int b = static_cast<int>(tile / p.rows_per_seq);
        const int hs = static_cast<int>(tile % p.rows_per_seq) / p.mt;
        const int kvh = p.per_qhead ? hs / p.g : hs;
        const int64_t plane = static_cast<int64_t>(b) * p.Hkv + kvh;
        const int len = tree_len(p, b);
        const int units = tree_units(p, len);
        const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
        if (reports && tile % p.rows_per_seq == 0 && unit == 0 && lane == 0 && p.len[b] != len)
            record_error(p.status, PISA_ERR_BAD_INDEX, kTreeDetail | 0xB0u);
        const int32_t* row = p.topk > 0 ? p.idx + (static_cast<int64_t>(b) * p.Hsel + hs) * p.topk : nullptr;
        const int nsel = p.topk * p.upb;
        const int uc = min(u1, units - 1);  // the last unit is the drafted tokens
        int first = -1;                     // a unit that waits for its partner
        for (int u = unit; u < uc && ok; u += 32) {
            int at = -1;  // position of this lane's unit; -1 = nothing there
            if (u + lane < uc) {
                const int c = u + lane;
                if (p.topk == 0) {
                    at = 64 * c;
                } else if (c >= nsel) {
                    at = p.seq + 64 * (c - nsel);
                } else {
                    const int j = __ldg(row + c / p.upb);
                    if (j >= p.n0) {
                        if (reports) record_error(p.status, PISA_ERR_BAD_INDEX, kTreeDetail | 0xB1u);
                    } else if (j >= 0) {
                        at = (j * p.upb + c % p.upb) * 64;
                    }
                }
            }
            for (uint32_t left = __ballot_sync(0xFFFFFFFFu, at >= 0 && at < len); left != 0 && ok; left &= left - 1) {
                const int a = __shfl_sync(0xFFFFFFFFu, at, __ffs(left) - 1);
                if (!PAIRS) {
                    issue(kTileCache, plane, len, a, -1);
                } else if (first < 0) {
                    first = a;
                } else {
                    issue(kTileCache, plane, len, first, a);
                    first = -1;
                }
            }
        }
        if (PAIRS && first >= 0 && ok) issue(kTileCache, plane, len, first, -1);
        if (u1 == units && ok) issue(kTileDraft, plane, len, 0, 0);
        if (ok) issue(kTileEnd, plane, len, 0, 0);
        pos += u1 - unit;
        unit = 0;
        ++tile;
    }
}

}  // namespace pisa
