// What the two kernels of the tree attention share: the cut of the work into runs, and small helpers.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
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

// ---------------------------------------------------------------- operands

// Shared-memory matrix descriptor; layout: 0 = none, 2 = 128-byte, 4 = 64-byte swizzle.
__device__ __forceinline__ uint64_t tree_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(layout) << 61);
}
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// Instruction descriptor for kind::f8f6f4: A e4m3, B e4m3 (0) or e5m2 (1), fp32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t idesc_f8(int n, int b_type, int a_mn, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(b_type) << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t cvt_e5m2x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
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
// Whether the barrier's phase of this parity has completed (no wait).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return r != 0;
}
// ---------------------------------------------------------------- the copies

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

// The producer warp of the kernels whose tiles are 128 keys (two units): keeps a ring of K tiles and one
// of V tiles full. Every entry (a tile, or the end of a piece) takes a K slot and describes itself in
// meta[entry % kTreeMeta]; a tile takes a V slot too. K and V of a cache tile: [128 rows], bf16 as D / 64
// column tiles of 128 bytes; of the drafted tokens: D / 64 column tiles of 64 rows.
template <int D, bool E4M3>
__device__ __forceinline__ void tree_producer(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                              const CUtensorMap& tmDK, const CUtensorMap& tmDV, uint8_t* ring,
                                              uint8_t* vring, uint8_t* exps, uint64_t* kfull, uint64_t* kempty,
                                              uint64_t* vfull, uint64_t* vempty, int4* meta, int64_t pos, int64_t end,
                                              int64_t tile, int unit) {
    constexpr int TILE = 128 * (E4M3 ? D : 2 * D), EXPS = E4M3 ? 256 : 0;
    const int lane = threadIdx.x & 31;
    RingAt k, v;
    bool ok = true;
    if (lane == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmDK);
        prefetch_tmap(&tmDV);
    }
    // one entry: a tile's K and then its V, or the end of a piece; of a tile of the cache the first
    // keys of its halves (second -1: absent)
    auto issue = [&](int kind, int64_t plane, int len, int a0, int a1) {
        if (lane == 0) {
            ok = k.n < p.nk || mbar_wait(&kempty[k.s], k.par ^ 1u, p.status, kTreeDetail | 0x01u);
            if (ok) {
                uint8_t* kt = ring + k.s * TILE;
                uint64_t* kb = &kfull[k.s];
                const int e = k.n % kTreeMeta;
                const int halves = a1 >= 0 ? 2 : 1;
                const int dbytes = p.tp * 2 * D, dy = static_cast<int>(plane * p.T);
                if (kind == kTileEnd) {
                    meta[e] = make_int4(kind, 0, 0, 0);
                    mbar_arrive(kb);
                } else if (kind == kTileDraft) {
                    meta[e] = make_int4(kind, 0, 0, 0);
                    mbar_arrive_expect_tx(kb, dbytes);
    #pragma unroll
                    for (int c = 0; c < D / 64; ++c) tma_load_2d(kt + c * 8192, &tmDK, 64 * c, dy, kb);
                } else {
                    meta[e] = make_int4(kind, min(64, len - a0), a1 >= 0 ? min(64, len - a1) : 0, 0);
                    mbar_arrive_expect_tx(kb, halves * (TILE + EXPS) / 2);
                    for (int h = 0; h < halves; ++h) {
                        const int64_t row = plane * p.cap + (h == 0 ? a0 : a1);
                        if constexpr (E4M3) {
                            tma_load_2d(kt + h * 64 * D, &tmK, 0, static_cast<int>(row), kb);
                            bulk_load(exps + e * 256 + h * 64, p.k_exp + row, 64, kb);
                            bulk_load(exps + e * 256 + 128 + h * 64, p.v_exp + row, 64, kb);
                        } else {
    #pragma unroll
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_2d(kt + c * 16384 + h * 8192, &tmK, 64 * c, static_cast<int>(row), kb);
                        }
                    }
                }
                k.next(p.nk);
                if (kind != kTileEnd) {
                    ok = v.n < p.nv || mbar_wait(&vempty[v.s], v.par ^ 1u, p.status, kTreeDetail | 0x02u);
                    if (ok) {
                        uint8_t* vt = vring + v.s * TILE;
                        uint64_t* vb = &vfull[v.s];
                        if (kind == kTileDraft) {
                            mbar_arrive_expect_tx(vb, dbytes);
    #pragma unroll
                            for (int c = 0; c < D / 64; ++c) tma_load_2d(vt + c * 8192, &tmDV, 64 * c, dy, vb);
                        } else {
                            mbar_arrive_expect_tx(vb, halves * TILE / 2);
                            for (int h = 0; h < halves; ++h) {
                                const int y = static_cast<int>(plane * p.cap + (h == 0 ? a0 : a1));
                                if constexpr (E4M3) {
                                    tma_load_2d(vt + h * 64 * D, &tmV, 0, y, vb);
                                } else {
    #pragma unroll
                                    for (int c = 0; c < D / 64; ++c)
                                        tma_load_2d(vt + c * 16384 + h * 8192, &tmV, 64 * c, y, vb);
                                }
                            }
                        }
                        v.next(p.nv);
                    }
                }
            }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    };
    while (pos < end && ok) {
        const int b = static_cast<int>(tile / p.rows_per_seq);
        const int hs = static_cast<int>(tile % p.rows_per_seq) / p.mt;
        const int kvh = p.per_qhead ? hs / p.g : hs;
        const int64_t plane = static_cast<int64_t>(b) * p.Hkv + kvh;
        const int len = tree_len(p, b);
        const int units = tree_units(p, len);
        const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
        if (tile % p.rows_per_seq == 0 && unit == 0 && lane == 0 && p.len[b] != len)
            record_error(p.status, PISA_ERR_BAD_INDEX, kTreeDetail | 0xB0u);
        const int32_t* row = p.topk > 0 ? p.idx + (static_cast<int64_t>(b) * p.Hsel + hs) * p.topk : nullptr;
        const int nsel = p.topk * p.upb;
        const int uc = min(u1, units - 1);  // the last unit is the drafted tokens
        int first = -1;                     // a unit that waits for its partner
        for (int u = unit; u < uc && ok; u += 32) {
            // up to 32 units at a time: position of each unit's first key, -1 = nothing there
            int at = -1;
            if (u + lane < uc) {
                const int c = u + lane;
                if (p.topk == 0) {
                    at = 64 * c;
                } else if (c >= nsel) {
                    at = p.seq + 64 * (c - nsel);
                } else {
                    const int j = __ldg(row + c / p.upb);
                    if (j >= p.n0)
                        record_error(p.status, PISA_ERR_BAD_INDEX, kTreeDetail | 0xB1u);
                    else if (j >= 0)
                        at = (j * p.upb + c % p.upb) * 64;
                }
            }
            for (uint32_t left = __ballot_sync(0xFFFFFFFFu, at >= 0 && at < len); left != 0 && ok; left &= left - 1) {
                const int a = __shfl_sync(0xFFFFFFFFu, at, __ffs(left) - 1);
                if (first < 0) {
                    first = a;
                } else {
                    issue(kTileCache, plane, len, first, a);
                    first = -1;
                }
            }
        }
        if (first >= 0 && ok) issue(kTileCache, plane, len, first, -1);
        if (u1 == units && ok) issue(kTileDraft, plane, len, 0, 0);
        if (ok) issue(kTileEnd, plane, len, 0, 0);
        pos += u1 - unit;
        unit = 0;
        ++tile;
    }
    // every copy lands before the block ends, also when another role gave up (earlier uses of a slot
    // were complete before it was filled again)
    if (lane == 0) {
        for (int i = 0; i < p.nk && i < k.n; ++i) {
            k.s = k.s == 0 ? p.nk - 1 : k.s - 1;
            if (k.s == p.nk - 1) k.par ^= 1u;
            if (!mbar_wait(&kfull[k.s], k.par, p.status, kTreeDetail | 0x03u)) break;
        }
        for (int i = 0; i < p.nv && i < v.n; ++i) {
            v.s = v.s == 0 ? p.nv - 1 : v.s - 1;
            if (v.s == p.nv - 1) v.par ^= 1u;
            if (!mbar_wait(&vfull[v.s], v.par, p.status, kTreeDetail | 0x04u)) break;
        }
    }
}

}  // namespace pisa
