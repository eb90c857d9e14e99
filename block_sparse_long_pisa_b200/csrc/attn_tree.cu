// Attention of a tree of drafted tokens over a K/V cache (one drafted token is plain decode).
//
//   rows   the T drafted tokens of the gh query heads that share a selection row: gh * T rows, cut
//          into row tiles of R (16 .. 128)
//   keys   the cache in units of 64 keys (selected blocks and tail, or all of it, up to the
//          sequence's length), two units to a tile of 128, and last the drafted tokens themselves,
//          masked by their ancestor bits
//   O = softmax(scale Q K^T) V with a running maximum and sum (fp32); no score leaves the SM
//
// Bound: the bytes of the cache that are read, each once per row tile (the row tiles of a sequence
// read them close together, from L2 after the first).
//
// Keys on the M side. Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T: the 128
// keys of a tile fill the M = 128 lanes of tcgen05.mma whatever the number of rows, which is N (16
// for a decode step: an MMA costs by N), K and V are the A operands straight from the tiles that
// TMA wrote (V as MN-major), and a softmax thread owns one key: its mask, its exponent bytes and its
// store of P are its own. The row maximum is the only thing that crosses lanes, so it is kept (in
// shared memory) until some score exceeds it by 2^kLazy: a tile normally needs one barrier with a
// vote, and only when the vote says so the maxima are found anew and O is rescaled in TMEM.
// (Rows on the M side with mma.sync, 16 rows a warp, took 144 us for a decode step over 64 caches of
// 128K rows, 64 selected 8-bit blocks, and 507 us for trees of 48 tokens over 8 ragged bf16 caches:
// converting 8-bit fragments was bound by issue, the bf16 rows by that instruction's rate.)
//
// e4m3 rows go into the MMA as they are (kind::f8f6f4, K = 32); what is not 8-bit is split:
//   * a row of Q is scaled by a power of two to a maximum in [224, 448) and taken as e4m3 (4
//     significant bits) + e5m2 (the remainder of bf16's 8 bits needs 3): exact for values down to
//     2^-14 of the row's largest, off by 2^-26 of it below;
//   * P, as fp16, is cut into three e5m2 terms: an e5m2 value is the upper byte of an fp16 one, so
//     t1 = upper byte of p, t2 of p - t1, t3 of p - t1 - t2: 9 bits or more (bf16 has 8), P at most
//     2^15, so a probability of 2^-18 of the row's largest still has them and one of 2^-28 counts;
//   * K's row exponent and Q's multiply the score in fp32; V's goes into P: P' = p 2^(e - 127 - u), O
//     in units of 2^u, u set by the largest V exponent so far.
// A bf16 cache takes P as bf16 (range of V); so do the drafted tokens, which are bf16 in both.
//
// Work split. Sequences have unlike lengths that only the device knows, so the units of all row
// tiles are laid end to end and cut into equal runs, one per CTA of a fixed grid; a run may end one
// row tile, hold whole ones and begin another. A row tile inside one run is finished there; one that
// crosses runs leaves partial (o, m, l) that attn_tree_merge_kernel joins in run order. Every CTA
// finds its run by summing the lengths itself: no scheduling pass, no atomics in any sum, and the
// same inputs give the same bits.
//
// CTA (two on an SM where shared memory allows): four softmax warps (thread = key = TMEM lane), a
// producer warp that keeps a ring of tiles in flight by TMA, and an MMA warp (TMEM allocation, one
// issuing lane). Order of the MMA lane: S(i+1), then P.V(i), so a tile's scores are formed while the
// softmax of the one before runs; S is double buffered.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pisa_device.cuh"

namespace pisa {

constexpr uint32_t kTreeDetail = kKernTree << 8;
constexpr int kTreeUMin = -100;  // smallest unit exponent of O (e4m3)
constexpr int kTreeMaxStages = 8;
enum : int { kTileEnd = 0, kTileCache = 1, kTileDraft = 2 };

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

__device__ __forceinline__ float pow2i(int e) {  // e in [-126, 127]
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
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
// Barrier over the softmax threads; true if `x` holds in any of them.
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() { named_bar_sync(1, 128); }

template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 32)
        tmem_ld32(taddr, r);
    else
        tmem_ld16(taddr, r);
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 32)
        tmem_st32(taddr, r);
    else
        tmem_st16(taddr, r);
}

// ---------------------------------------------------------------- layout

template <int D, bool E4M3, int R>
struct TreeCfg {
    static constexpr int ROW = E4M3 ? D : 2 * D;         // bytes of a cache row
    static constexpr int TILE = 128 * ROW;               // K (or V) of one tile
    static constexpr int STAGE = 2 * TILE;
    static constexpr int EXPS = E4M3 ? 256 : 0;          // a stage's exponent bytes of K and of V
    static constexpr int QB = R * 2 * D;                 // Q: bf16, or the e4m3 and the e5m2 terms
    static constexpr int PTERM = R * 128;                // one 8-bit term of P
    static constexpr int PB = E4M3 ? 3 * PTERM : 2 * PTERM;
    // P buffers: one where a second would cost a CTA per SM (e4m3, 64 rows) or a stage (bf16, many rows)
    static constexpr int NP = (E4M3 ? R == 64 : R > 64) ? 1 : 2;
    static constexpr int CW = R < 32 ? 16 : 32;          // TMEM columns taken at a time
    static constexpr int COLS = 3 * R <= 64 ? 64 : 3 * R <= 128 ? 128 : 3 * R <= 256 ? 256 : 512;
    static constexpr float LAZY = E4M3 ? 4.f : 8.f;      // log2 units a score may exceed the kept maximum by
    // dynamic shared memory without the ring: Q, P, masks, row parameters (8 floats a row)
    static constexpr int FIXED = 1024 + QB + NP * PB + R * 8 + R * 32;
    static constexpr int CTAS = E4M3 && R <= 64 ? 2 : 1;  // CTAs an SM's shared memory takes
};

template <int D, bool E4M3, int R>
__global__ void __launch_bounds__(192, TreeCfg<D, E4M3, R>::CTAS)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                     const TreeParams p) {
    using C = TreeCfg<D, E4M3, R>;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* q_s = ring + p.nstg * C::STAGE;
    uint8_t* p_s = q_s + C::QB;
    uint64_t* mask_s = reinterpret_cast<uint64_t*>(p_s + C::NP * C::PB);  // [R]
    float* rf_s = reinterpret_cast<float*>(mask_s + R);  // score factor of a row (e4m3: 2^-(Q's exponent))
    float* nm_s = rf_s + R;                              // -(kept maximum), 0 while there is none
    float* m_s = nm_s + R;                               // kept maximum, log2 units
    float* al_s = m_s + R;                               // factor of O and l in a rescale; 1/l at the end
    float* w_s = al_s + R;                               // [4 warps][R]
    uint8_t* exps = reinterpret_cast<uint8_t*>(w_s + 4 * R);  // [stage][K 128, V 128]
    __shared__ __align__(8) uint64_t full[kTreeMaxStages], empty[kTreeMaxStages], sfull[2], pfull[2], pvdone[2], qfull, done;
    __shared__ int4 meta[kTreeMaxStages];  // kind, keys that count in the two halves
    __shared__ uint32_t tmem_slot, dflag[2], wexp[4];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const TreeJob job = tree_job(p);
    if (static_cast<int64_t>(blockIdx.x) >= job.runs) return;
    int64_t pos = job.begin(blockIdx.x);
    const int64_t end = job.begin(blockIdx.x + 1);
    int64_t tile;
    int unit;
    tree_find(p, pos, tile, unit);
    if (tid == 0) {
        for (int i = 0; i < p.nstg; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 5);  // the softmax warps, and P.V (or the MMA lane itself)
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&pvdone[i], 1);
        }
        mbar_init(&qfull, 4);
        mbar_init(&done, 1);
        fence_barrier_init();
    }
    if (warp == 5) tmem_alloc(&tmem_slot, C::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    const uint32_t tm_o = tm + 2 * R;

    int s = 0;            // ring stage, and the parity of its current use
    uint32_t par = 0;
    bool ok = true;       // cleared by a wait that ran out: nothing more is waited for
    auto advance = [&]() {
        if (++s == p.nstg) {
            s = 0;
            par ^= 1u;
        }
    };
    const int dtile = D * 128;  // drafted K (or V) in a stage: [D / 64][64 rows][128 B]

    if (warp == 4) {
        // ------------------------------------------------ producer
        int used = 0;   // ring slots handed out
        if (lane == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            prefetch_tmap(&tmDK);
            prefetch_tmap(&tmDV);
        }
        // one slot: kind, and for a tile the first keys of its halves (second -1: absent)
        auto issue = [&](int kind, int64_t plane, int len, int a0, int a1) {
            if (lane == 0) {
                ok = used < p.nstg || mbar_wait(&empty[s], par ^ 1u, p.status, kTreeDetail | 0x01u);
                if (ok) {
                    uint8_t* kt = ring + s * C::STAGE;
                    if (kind == kTileEnd) {
                        meta[s] = make_int4(kind, 0, 0, 0);
                        mbar_arrive(&full[s]);
                    } else if (kind == kTileDraft) {
                        meta[s] = make_int4(kind, 0, 0, 0);
                        mbar_arrive_expect_tx(&full[s], 2 * p.tp * 2 * D);
                        const int y = static_cast<int>(plane * p.T);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            tma_load_2d(kt + c * 8192, &tmDK, 64 * c, y, &full[s]);
                            tma_load_2d(kt + dtile + c * 8192, &tmDV, 64 * c, y, &full[s]);
                        }
                    } else {
                        const int halves = a1 >= 0 ? 2 : 1;
                        meta[s] = make_int4(kind, min(64, len - a0), a1 >= 0 ? min(64, len - a1) : 0, 0);
                        mbar_arrive_expect_tx(&full[s], halves * (C::STAGE + C::EXPS) / 2);
                        for (int h = 0; h < halves; ++h) {
                            const int64_t row = plane * p.cap + (h == 0 ? a0 : a1);
                            const int y = static_cast<int>(row);
                            if constexpr (E4M3) {
                                tma_load_2d(kt + h * 64 * D, &tmK, 0, y, &full[s]);
                                tma_load_2d(kt + C::TILE + h * 64 * D, &tmV, 0, y, &full[s]);
                                bulk_load(exps + s * 256 + h * 64, p.k_exp + row, 64, &full[s]);
                                bulk_load(exps + s * 256 + 128 + h * 64, p.v_exp + row, 64, &full[s]);
                            } else {
#pragma unroll
                                for (int c = 0; c < D / 64; ++c) {
                                    tma_load_2d(kt + c * 16384 + h * 8192, &tmK, 64 * c, y, &full[s]);
                                    tma_load_2d(kt + C::TILE + c * 16384 + h * 8192, &tmV, 64 * c, y, &full[s]);
                                }
                            }
                        }
                    }
                }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (ok) {
                ++used;
                advance();
            }
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
        // every copy lands before the block ends, also when another role gave up (earlier uses of a
        // stage were complete before it was filled again)
        if (lane == 0) {
            for (int i = 0; i < p.nstg && i < used; ++i) {
                s = s == 0 ? p.nstg - 1 : s - 1;
                if (s == p.nstg - 1) par ^= 1u;
                if (!mbar_wait(&full[s], par, p.status, kTreeDetail | 0x02u)) break;
            }
        }
    } else if (warp == 5) {
        // ------------------------------------------------ MMA
        if (lane == 0) {
            const uint32_t q0 = smem_u32(q_s), p0 = smem_u32(p_s);
            int it = 0;               // tiles so far
            uint32_t qpar = 0;
            bool issued = false;
            int pend_s = -1, pend_kind = 0;
            bool fresh = true;        // the next P.V begins O
            auto pv = [&]() {         // P.V of the tile before (number it - 1 when called)
                const int j = it - 1;
                ok = mbar_wait(&pfull[j & 1], (j >> 1) & 1, p.status, kTreeDetail | 0x03u);
                if (!ok) return;
                tc_fence_after();
                const uint32_t pb = p0 + (j % C::NP) * C::PB;
                const uint32_t vt = smem_u32(ring + pend_s * C::STAGE);
                if (pend_kind == kTileDraft || !E4M3) {
                    const bool draft = pend_kind == kTileDraft;
                    const uint32_t sub = draft ? 8192 : 16384;
                    const uint64_t a = tree_desc(vt + (draft ? dtile : C::TILE), D == 128 ? sub : 0, 1024, 2);
                    const uint64_t b = tree_desc(pb, 128, 2048, 0);
                    const int steps = draft ? p.tp / 16 : 8;
                    for (int k = 0; k < steps; ++k)
                        mma_bf16_ss(tm_o, desc_at(a, k * 2048), desc_at(b, k * 256), idesc_bf16_f32(128, R, 1, 1),
                                    !fresh || k > 0 ? 1u : 0u);
                } else {
                    const uint64_t a = D == 128 ? tree_desc(vt + C::TILE, 0, 1024, 2) : tree_desc(vt + C::TILE, 0, 512, 4);
                    const uint64_t b = tree_desc(pb, 128, 2048, 0);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int t = 0; t < 3; ++t)
                            mma_f8_ss(tm_o, desc_at(a, k * 32 * D), desc_at(b, t * C::PTERM + k * 512), idesc_f8(R, 1, 1, 1),
                                      !fresh || k > 0 || t > 0 ? 1u : 0u);
                    }
                }
                fresh = false;
                mma_commit(&empty[pend_s]);
                mma_commit(&pvdone[j % C::NP]);
            };
            while (pos < end && ok) {
                const int b = static_cast<int>(tile / p.rows_per_seq);
                const int units = tree_units(p, tree_len(p, b));
                const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
                fresh = true;
                bool first = true;
                while (ok) {
                    ok = mbar_wait(&full[s], par, p.status, kTreeDetail | 0x05u);
                    if (!ok) break;
                    const int kind = meta[s].x;
                    if (kind == kTileEnd) {
                        if (pend_s >= 0) pv();
                        pend_s = -1;
                        if (ok) {
                            mbar_arrive(&empty[s]);
                            advance();
                        }
                        break;
                    }
                    if (first || (E4M3 && kind == kTileDraft)) {  // for the drafted tokens Q comes again, as bf16
                        ok = mbar_wait(&qfull, qpar, p.status, kTreeDetail | 0x06u);
                        qpar ^= 1u;
                        first = false;
                        if (!ok) break;
                    }
                    tc_fence_after();
                    const uint32_t kt = smem_u32(ring + s * C::STAGE);
                    const uint32_t d = tm + (it & 1) * R;
                    issued = true;
                    if (kind == kTileDraft || !E4M3) {
                        const uint32_t sub = kind == kTileDraft ? 8192 : 16384;
                        const uint64_t a = tree_desc(kt, 16, 1024, 2), bq = tree_desc(q0, 16, 1024, 2);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_bf16_ss(d, desc_at(a, (k / 4) * sub + (k % 4) * 32), desc_at(bq, (k / 4) * (R * 128) + (k % 4) * 32),
                                        idesc_bf16_f32(128, R, 0, 0), k > 0 ? 1u : 0u);
                    } else {
                        const uint64_t a = D == 128 ? tree_desc(kt, 16, 1024, 2) : tree_desc(kt, 16, 512, 4);
                        const uint64_t bq = D == 128 ? tree_desc(q0, 16, 1024, 2) : tree_desc(q0, 16, 512, 4);
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            mma_f8_ss(d, desc_at(a, k * 32), desc_at(bq, k * 32), idesc_f8(R, 0, 0, 0), k > 0 ? 1u : 0u);
                            mma_f8_ss(d, desc_at(a, k * 32), desc_at(bq, R * D + k * 32), idesc_f8(R, 1, 0, 0), 1u);
                        }
                    }
                    mma_commit(&sfull[it & 1]);
                    if (pend_s >= 0) pv();
                    pend_s = s;
                    pend_kind = kind;
                    ++it;
                    advance();
                }
                pos += u1 - unit;
                unit = 0;
                ++tile;
            }
            if (issued) {  // nothing of this CTA's still runs when TMEM goes
                mma_commit(&done);
                mbar_wait(&done, 0, p.status, kTreeDetail | 0x07u);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax: thread = key of the tile = TMEM lane
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;  // TMEM lane base of the warp
        const int rows = p.gh * p.T;
        int it = 0;
        while (pos < end && ok) {
            const int b = static_cast<int>(tile / p.rows_per_seq);
            const int rem = static_cast<int>(tile % p.rows_per_seq);
            const int hs = rem / p.mt, row_base = (rem % p.mt) * R;
            const int units = tree_units(p, tree_len(p, b));
            const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
            const int64_t out0 = (static_cast<int64_t>(b) * p.Hq + hs * p.gh) * p.T;  // first row of the group
            const int nrows = min(R, rows - row_base);
            const uint4* qg = reinterpret_cast<const uint4*>(p.Q + (out0 + row_base) * D);

            // Q as bf16: [D / 64][R rows][128 B], 128-byte swizzle
            auto q_bf16 = [&]() {
                for (int e = tid; e < R * (D / 8); e += 128) {
                    const int r = e / (D / 8), c = e % (D / 8);
                    const uint4 x = r < nrows ? __ldg(qg + e) : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(q_s + (c / 8) * (R * 128) + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = x;
                }
            };
            // Q as e4m3 + e5m2 terms [R rows][D B], swizzled by the row's size; D/8 lanes hold a row
            auto q_terms = [&]() {
                for (int e = tid; e < R * (D / 8); e += 128) {  // R * D / 8 is a multiple of 128
                    const int r = e / (D / 8), c = e % (D / 8);
                    const uint4 x = r < nrows ? __ldg(qg + e) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    float v[8], top = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        v[k] = __uint_as_float((k & 1) ? (w[k / 2] & 0xFFFF0000u) : (w[k / 2] << 16));
                        top = fmaxf(top, fabsf(v[k]));
                    }
#pragma unroll
                    for (int o = 1; o < D / 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    // 2^(f - 127) brings the maximum to [224, 448): 448 = 1.75 * 2^8
                    const uint32_t tb = __float_as_uint(top);
                    const int f = min(253, 127 + 8 + 127 - static_cast<int>(tb >> 23) - ((tb & 0x7FFFFFu) > 0x600000u ? 1 : 0));
                    const float sc = __uint_as_float(static_cast<uint32_t>(f) << 23);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float a = v[2 * k] * sc, bb = v[2 * k + 1] * sc;
                        hi[k] = cvt_e4m3x2(a, bb);
                        const float2 h = e4m3x2_f32(hi[k]);
                        // an infinity saturates: its remainder keeps it (inf - 448) as a NaN
                        lo[k] = cvt_e5m2x2(a - h.x, bb - h.y);
                        if (isinf(a)) lo[k] = (lo[k] & 0xFF00u) | 0x7Fu;
                        if (isinf(bb)) lo[k] = (lo[k] & 0x00FFu) | 0x7F00u;
                    }
                    const int ch = c / 2;  // 16-byte chunk of the row
                    const uint32_t off = D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) + 8 * (c & 1)
                                                  : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4) + 8 * (c & 1);
                    *reinterpret_cast<uint2*>(q_s + off) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                    *reinterpret_cast<uint2*>(q_s + R * D + off) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
                    if (c == 0) rf_s[r] = __uint_as_float(static_cast<uint32_t>(254 - f) << 23);
                }
            };
            auto q_ready = [&]() {  // this warp's part of it
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull);
            };
            if constexpr (E4M3)
                q_terms();
            else
                q_bf16();
            if (u1 == units && tid < R) {  // this piece ends with the drafted tokens
                const int rg = row_base + tid;
                const uint64_t live = p.T == 64 ? ~0ull : (1ull << p.T) - 1ull;
                mask_s[tid] = rg < rows ? __ldg(p.mask + static_cast<int64_t>(b) * p.T + rg % p.T) & live : 0ull;
            }
            if (tid < 2) dflag[tid] = 0;
            softmax_sync();  // row factors and masks

            uint64_t l2[R / 2];  // this key's share of the rows' sums
#pragma unroll
            for (int i = 0; i < R / 2; ++i) l2[i] = 0ull;
            bool fresh = true;
            int u = 0, uexp = 0;   // unit exponent of O, and the V exponent it was set by (e4m3)

            while (true) {
                // Every slot is one barrier, and a second one when the first says so: a warp whose wait ran
                // out takes both, so that all warps leave together whatever the others saw in the slot.
                if (ok) ok = mbar_wait(&full[s], par, p.status, kTreeDetail | 0x08u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                const int4 mt = ok ? meta[s] : make_int4(kTileEnd, 0, 0, 0);
                if (mt.x == kTileEnd) {
                    if (softmax_any(!ok) && softmax_any(!ok)) ok = false;
                    if (ok) {
                        if (lane == 0) mbar_arrive(&empty[s]);
                        advance();
                    }
                    break;
                }
                const bool draft = mt.x == kTileDraft;
                // Q is handed over at the first tile, not before it is known that there is one: a piece may
                // hold no tile at all, and its successor's Q must not be announced before the MMA lane
                // has seen this one's
                if (E4M3 && draft) {
                    q_bf16();  // every S of this piece so far is formed: Q's buffer is free
                    q_ready();
                } else if (fresh) {
                    q_ready();
                }
                uint8_t* kt = ring + s * C::STAGE;
                const bool valid = draft ? tid < p.T : (tid & 63) < (tid < 64 ? mt.y : mt.z);
                const bool partial = draft || mt.y < 64 || mt.z < 64;
                float kf = p.scale_log2;
                int ev = 0;
                if (E4M3 && !draft && valid) {
                    kf *= __uint_as_float(static_cast<uint32_t>(exps[s * 256 + tid]) << 23);
                    ev = exps[s * 256 + 128 + tid];
                }
                ok = __all_sync(0xFFFFFFFFu, ok) && mbar_wait(&sfull[it & 1], (it >> 1) & 1, p.status, kTreeDetail | 0x09u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                tc_fence_after();
                const uint32_t ts = tm + lanes + (it & 1) * R;
                const uint64_t kf2 = f2_pack(kf, kf);

                // scores against the kept maximum, log2 units, of columns [c0, c0 + CW)
                auto load_scores = [&](int c0, uint64_t (&x)[C::CW / 2], bool against) {
                    uint32_t v[C::CW];
                    tmem_ldn<C::CW>(ts + c0, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < C::CW / 4; ++i) {
                        const float4 nm = *reinterpret_cast<const float4*>(nm_s + c0 + 4 * i);
                        uint64_t a = f2_mul(f2_pack(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), kf2);
                        uint64_t c = f2_mul(f2_pack(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), kf2);
                        uint64_t ma = f2_pack(nm.x, nm.y), mc = f2_pack(nm.z, nm.w);
                        if (!against) ma = mc = 0ull;
                        if constexpr (E4M3) {
                            float4 rf = *reinterpret_cast<const float4*>(rf_s + c0 + 4 * i);
                            if (draft) rf = make_float4(1.f, 1.f, 1.f, 1.f);  // bf16 rows as they are
                            a = f2_fma(a, f2_pack(rf.x, rf.y), ma);
                            c = f2_fma(c, f2_pack(rf.z, rf.w), mc);
                        } else {
                            a = f2_add(a, ma);
                            c = f2_add(c, mc);
                        }
                        x[2 * i] = a;
                        x[2 * i + 1] = c;
                    }
                    if (draft) {
#pragma unroll
                        for (int i = 0; i < C::CW / 2; ++i) {
                            float lo, hi;
                            f2_unpack(x[i], lo, hi);
                            lo = valid && (mask_s[c0 + 2 * i] >> tid) & 1ull ? lo : -INFINITY;
                            hi = valid && (mask_s[c0 + 2 * i + 1] >> tid) & 1ull ? hi : -INFINITY;
                            x[i] = f2_pack(lo, hi);
                        }
                    }
                };
                float top = -INFINITY;
                if (!fresh) {
                    for (int c0 = 0; c0 < R; c0 += C::CW) {
                        uint64_t x[C::CW / 2];
                        load_scores(c0, x, true);
#pragma unroll
                        for (int i = 0; i < C::CW / 2; ++i) {
                            float lo, hi;
                            f2_unpack(x[i], lo, hi);
                            top = fmax3(top, lo, hi);
                        }
                    }
                }
                const bool over = valid && (top > C::LAZY || (E4M3 && !draft && ev > uexp));
                if (softmax_any(!ok || fresh || over)) {
                    if (softmax_any(!ok)) {
                        ok = false;
                        break;
                    }
                    // the rows' maxima over this tile, and the largest V exponent
                    for (int c0 = 0; c0 < R; c0 += C::CW) {
                        uint64_t x[C::CW / 2];
                        load_scores(c0, x, false);
                        float mine = -INFINITY;
#pragma unroll
                        for (int i = 0; i < C::CW / 2; ++i) {
                            float lo, hi;
                            f2_unpack(x[i], lo, hi);
                            lo = warp_max(valid ? lo : -INFINITY);
                            hi = warp_max(valid ? hi : -INFINITY);
                            if (lane == 2 * i) mine = lo;
                            if (lane == 2 * i + 1) mine = hi;
                        }
                        if (lane < C::CW) w_s[warp * R + c0 + lane] = mine;
                    }
                    if constexpr (E4M3) {
                        const uint32_t we = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(ev));
                        if (lane == 0) wexp[warp] = we;
                    }
                    softmax_sync();
                    if (tid < R) {
                        const float M = fmaxf(fmaxf(w_s[tid], w_s[R + tid]), fmaxf(w_s[2 * R + tid], w_s[3 * R + tid]));
                        const float old = fresh ? -INFINITY : m_s[tid];
                        const float now = fmaxf(old, M);
                        al_s[tid] = now == old ? 1.f : fast_exp2(old - now);
                        m_s[tid] = now;
                        nm_s[tid] = now == -INFINITY ? 0.f : -now;
                    }
                    float uf = 1.f;
                    if (E4M3 && !draft) {
                        const int e = static_cast<int>(min(254u, max(max(wexp[0], wexp[1]), max(wexp[2], wexp[3]))));
                        if (fresh || e > uexp) {
                            uexp = e;
                            const int un = max(kTreeUMin, e - 127 + static_cast<int>(C::LAZY) - 15);
                            uf = pow2i(max(-126, u - un));  // u - un <= 0 once O holds anything
                            u = un;
                        }
                    }
                    softmax_sync();
                    if (!fresh) {
                        const int j = it - 1;
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pvdone[j % C::NP], (j / C::NP) & 1, p.status,
                                                               kTreeDetail | 0x0Au));
                        tc_fence_after();
                        for (int c0 = 0; c0 < R; c0 += C::CW) {
                            uint32_t v[C::CW];
                            tmem_ldn<C::CW>(tm_o + lanes + c0, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < C::CW; ++i)
                                v[i] = __float_as_uint(__uint_as_float(v[i]) * (al_s[c0 + i] * uf));
                            tmem_stn<C::CW>(tm_o + lanes + c0, v);
                        }
                        tmem_wait_st();
#pragma unroll
                        for (int i = 0; i < R / 2; ++i) l2[i] = f2_mul(l2[i], f2_pack(al_s[2 * i], al_s[2 * i + 1]));
                    }
                    fresh = false;
                }
                // P's buffer: the P.V that read it last is complete
                if (it >= C::NP && ok) {
                    const int j = it - C::NP;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pvdone[j % C::NP], (j / C::NP) & 1, p.status,
                                                           kTreeDetail | 0x0Bu));
                }
                uint8_t* pb = p_s + (it % C::NP) * C::PB;
                // a row of exponent 255 stands for NaN (its bytes are zero)
                const float pf = !E4M3 ? 1.f
                                 : draft ? pow2i(min(127, max(-126, -u)))
                                         : __uint_as_float(ev == 255 ? 0x7FFFFFFFu : static_cast<uint32_t>(max(ev - u, 0)) << 23);
                const uint64_t pf2 = f2_pack(pf, pf);
#pragma unroll
                for (int c0 = 0; c0 < R; c0 += C::CW) {
                    uint64_t x[C::CW / 2];
                    load_scores(c0, x, true);
                    float pr[C::CW];
#pragma unroll
                    for (int i = 0; i < C::CW / 2; ++i) {
                        float lo, hi;
                        f2_unpack(x[i], lo, hi);
                        pr[2 * i] = fast_exp2(lo);
                        pr[2 * i + 1] = fast_exp2(hi);
                    }
                    if (partial) {
#pragma unroll
                        for (int i = 0; i < C::CW; ++i) pr[i] = valid ? pr[i] : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < C::CW / 2; ++i) {
                        x[i] = f2_pack(pr[2 * i], pr[2 * i + 1]);
                        l2[c0 / 2 + i] = f2_add(l2[c0 / 2 + i], x[i]);
                        if constexpr (E4M3) x[i] = f2_mul(x[i], pf2);
                    }
                    if (partial && E4M3) {
#pragma unroll
                        for (int i = 0; i < C::CW / 2; ++i) x[i] = valid ? x[i] : 0ull;
                    }
                    if (E4M3 && !draft) {
#pragma unroll
                        for (int g = 0; g < C::CW / 16; ++g) {
                            uint32_t t1[4], t2[4], t3[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t h[2], a1[2], a2[2], a3[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    float lo, hi;
                                    f2_unpack(x[8 * g + 2 * k + e], lo, hi);
                                    h[e] = pack_f16x2(lo, hi);
                                    a1[e] = h[e] & 0xFF00FF00u;
                                    h[e] = sub_f16x2(h[e], a1[e]);
                                    a2[e] = h[e] & 0xFF00FF00u;
                                    a3[e] = sub_f16x2(h[e], a2[e]) + 0x00800080u;  // rounded, not cut
                                }
                                t1[k] = __byte_perm(a1[0], a1[1], 0x7531);
                                t2[k] = __byte_perm(a2[0], a2[1], 0x7531);
                                t3[k] = __byte_perm(a3[0], a3[1], 0x7531);
                            }
                            uint8_t* dst = pb + (c0 / 16 + g) * 2048 + tid * 16;
                            *reinterpret_cast<uint4*>(dst) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                            *reinterpret_cast<uint4*>(dst + C::PTERM) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
                            *reinterpret_cast<uint4*>(dst + 2 * C::PTERM) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
                        }
                    } else {
#pragma unroll
                        for (int g = 0; g < C::CW / 8; ++g) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float lo, hi;
                                f2_unpack(x[4 * g + k], lo, hi);
                                w[k] = pack_bf16x2(lo, hi);
                            }
                            *reinterpret_cast<uint4*>(pb + (c0 / 8 + g) * 2048 + tid * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (partial && !valid && !draft) {
                    // what the cache holds past the sequence must not meet P's zeros as a NaN
                    for (int c = 0; c < C::ROW / 16; ++c) {
                        uint8_t* v = kt + C::TILE + (E4M3 ? tid * D + 16 * c : (c / 8) * 16384 + tid * 128 + 16 * (c % 8));
                        *reinterpret_cast<uint4*>(v) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                if (draft && tid < p.tp) {
                    // a drafted value that is not finite would reach every token through 0 * x: it is taken
                    // out here and given to the tokens that attend it at the end
                    uint32_t bad = 0;
                    for (int c = 0; c < D / 8; ++c) {
                        uint4* v = reinterpret_cast<uint4*>(kt + dtile + (c / 8) * 8192 + tid * 128 + 16 * (c % 8));
                        uint32_t w[4] = {v->x, v->y, v->z, v->w};
                        uint32_t any = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((w[k] & 0x7F80u) == 0x7F80u) w[k] &= 0xFFFF0000u, any = 1;
                            if ((w[k] & 0x7F800000u) == 0x7F800000u) w[k] &= 0x0000FFFFu, any = 1;
                        }
                        if (!valid) {
                            *v = make_uint4(0u, 0u, 0u, 0u);
                        } else if (any) {
                            *v = make_uint4(w[0], w[1], w[2], w[3]);
                            bad = 1;
                        }
                    }
                    if (bad) atomicOr(&dflag[tid >> 5], 1u << (tid & 31));
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&pfull[it & 1]);
                    mbar_arrive(&empty[s]);
                }
                ++it;
                advance();
            }
            if (!ok) break;

            // ---- the piece's end: sums over the keys, then O^T (lane = dim) to its rows
            const bool any_tile = !fresh;
            for (int c0 = 0; c0 < R; c0 += C::CW) {
                float v[C::CW];
#pragma unroll
                for (int i = 0; i < C::CW / 2; ++i) {
                    // constant register indices: pick the chunk by selects the compiler folds
                    uint64_t x = 0ull;
#pragma unroll
                    for (int cc = 0; cc < R / C::CW; ++cc)
                        if (cc * C::CW == c0) x = l2[cc * (C::CW / 2) + i];
                    f2_unpack(x, v[2 * i], v[2 * i + 1]);
                }
                // lane j ends with the sum of column j: halves are exchanged, the kept half is added
                int n = C::CW;
                if constexpr (C::CW == 32) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const bool up = lane & 16;
                        const float give = up ? v[i] : v[i + 16], keep = up ? v[i + 16] : v[i];
                        v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 16);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 16);
                }
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (i >= o) break;
                        const bool up = lane & o;
                        const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
                        v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                    }
                }
                if (lane < n) w_s[warp * R + c0 + lane] = v[0];
            }
            softmax_sync();
            const bool whole = unit == 0 && u1 == units;
            // partial slots: 2c for a piece that goes on with a row tile, 2c + 1 for one that begins it
            float* part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (unit == 0 ? 1 : 0)) * R * (D + 2);
            if (tid < R) {
                const float l = (w_s[tid] + w_s[R + tid]) + (w_s[2 * R + tid] + w_s[3 * R + tid]);
                const float m = any_tile ? m_s[tid] : -INFINITY;
                al_s[tid] = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                if (whole) {
                    if (p.lse != nullptr && tid < nrows)
                        p.lse[out0 + row_base + tid] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                } else {
                    part[R * D + 2 * tid] = l == 0.f ? -INFINITY : m;
                    part[R * D + 2 * tid + 1] = l;
                }
            }
            softmax_sync();
            if (any_tile) {
                const int j = it - 1;
                ok = mbar_wait(&pvdone[j % C::NP], (j / C::NP) & 1, p.status, kTreeDetail | 0x0Cu);
                tc_fence_after();
            }
            const float uf = E4M3 ? pow2i(min(127, max(-126, u))) : 1.f;
            const uint64_t odd = dflag[0] | (static_cast<uint64_t>(dflag[1]) << 32);
            const int kvh = p.per_qhead ? hs / p.g : hs;
            for (int c0 = 0; c0 < R; c0 += C::CW) {
                if (c0 >= nrows) break;
                uint32_t v[C::CW];
                if (any_tile) {
                    tmem_ldn<C::CW>(tm_o + lanes + c0, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < C::CW; ++i) v[i] = 0u;
                }
                if (tid < D) {
#pragma unroll
                    for (int i = 0; i < C::CW; ++i) {
                        const int r = c0 + i;
                        if (r < nrows) {
                            float x = __uint_as_float(v[i]) * (uf * al_s[r]);
                            if (odd != 0) {
                                for (uint64_t left = odd & mask_s[r]; left != 0; left &= left - 1) {
                                    const int jd = __ffsll(static_cast<long long>(left)) - 1;
                                    const float y = __bfloat162float(
                                        p.DV[((static_cast<int64_t>(b) * p.Hkv + kvh) * p.T + jd) * D + tid]);
                                    if (!isfinite(y)) x += y;
                                }
                            }
                            if (whole)
                                p.O[(out0 + row_base + r) * D + tid] = __float2bfloat16_rn(x);
                            else
                                part[r * D + tid] = x;
                        }
                    }
                }
            }
            tc_fence_before();
            if (softmax_any(!ok)) ok = false;  // row parameters are free for the next piece
            pos += u1 - unit;
            unit = 0;
            ++tile;
        }
    }
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tm, C::COLS);
    }
}

// Joins the pieces of the row tiles that crossed runs, in run order: m = max m_i, weights
// 2^(m_i - m). grid: (row tiles, groups of four rows); 128 threads, one float4 of a row each (D = 128).
template <int D>
__global__ void __launch_bounds__(128) attn_tree_merge_kernel(const TreeParams p, int RM) {
    const int64_t tile = blockIdx.x;
    const int b = static_cast<int>(tile / p.rows_per_seq);
    const int rem = static_cast<int>(tile % p.rows_per_seq);
    const int hs = rem / p.mt, row_base = (rem % p.mt) * RM;
    const int rows = p.gh * p.T;
    const int row = static_cast<int>(blockIdx.y) * 4 + static_cast<int>(threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row_base + row >= rows) return;
    const TreeJob job = tree_job(p);
    // units before this row tile (whole warp)
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int i = lane; i < b; i += 32) before += tree_units(p, tree_len(p, i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    const int units = tree_units(p, tree_len(p, b));
    const int64_t x0 = before * p.rows_per_seq + static_cast<int64_t>(rem) * units;
    const int64_t c0 = job.run_of(x0), c1 = job.run_of(x0 + units - 1);
    if (c0 == c1) return;
    const int64_t stride = static_cast<int64_t>(RM) * (D + 2);
    auto slot = [&](int64_t c) { return p.part + (2 * c + (c == c0 ? 1 : 0)) * stride; };
    float M = -INFINITY;
    for (int64_t c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, slot(c)[RM * D + 2 * row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    constexpr int V = D / 32;  // values of the row per lane
    float acc[V], l = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int64_t c = c0; c <= c1; ++c) {
        const float* s = slot(c);
        const float mc = s[RM * D + 2 * row], lc = s[RM * D + 2 * row + 1];
        const float w = mc == -INFINITY ? (lc == 0.f ? 0.f : 1.f) : fast_exp2(mc - M);
        float v[V];
        if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4*>(s + row * D + 4 * lane);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2*>(s + row * D + 2 * lane);
            v[0] = x.x, v[1] = x.y;
        }
        l += w * lc;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += w * v[k];
    }
    const int64_t orow = (static_cast<int64_t>(b) * p.Hq + hs * p.gh) * p.T + row_base + row;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if constexpr (V == 4)
        *reinterpret_cast<uint2*>(p.O + orow * D + 4 * lane) =
            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t*>(p.O + orow * D + 2 * lane) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}

// ---------------------------------------------------------------- host side

// Rows of one row tile for a selection row of `rows` rows: the smallest of 16, 32, 64, 96 and 128 that
// holds them, or, past 128 rows, of 96 and 128 the one that pads less (128 on a tie).
int tree_row_tile(int rows) {
    for (int r : {16, 32, 64, 96, 128})
        if (rows <= r) return r;
    return (rows + 95) / 96 * 96 < (rows + 127) / 128 * 128 ? 96 : 128;
}

// CTAs on one SM: two where the shared memory of both fits.
int tree_ctas_per_sm(int rm, bool e4m3) { return e4m3 && rm <= 64 ? 2 : 1; }

template <int D, bool E4M3, int R>
static bool launch_tree(TreeParams p, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dk,
                        const CUtensorMap& dv, cudaStream_t st, int32_t* launches) {
    using C = TreeCfg<D, E4M3, R>;
    constexpr int budget = (C::CTAS == 2 ? 112 : 225) * 1024;
    static_assert(C::FIXED + 2 * (C::STAGE + C::EXPS) <= budget, "two stages must fit");
    p.nstg = (budget - C::FIXED) / (C::STAGE + C::EXPS);
    if (p.nstg > kTreeMaxStages) p.nstg = kTreeMaxStages;
    const int smem = C::FIXED + p.nstg * (C::STAGE + C::EXPS);
    static std::atomic<uint64_t> configured{0};
    if (!configure_smem_once(reinterpret_cast<const void*>(attn_tree_kernel<D, E4M3, R>), smem, configured)) return false;
    attn_tree_kernel<D, E4M3, R><<<p.runs, 192, smem, st>>>(k, v, dk, dv, p);
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.rows_per_seq, R / 4);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, attn_tree_merge_kernel<D>, p, R) != cudaSuccess) return false;
    ++*launches;
    return true;
}

template <int D, bool E4M3>
static bool launch_tree_rows(const TreeParams& p, int rm, const CUtensorMap& k, const CUtensorMap& v,
                             const CUtensorMap& dk, const CUtensorMap& dv, cudaStream_t st, int32_t* launches) {
    switch (rm) {
        case 16: return launch_tree<D, E4M3, 16>(p, k, v, dk, dv, st, launches);
        case 32: return launch_tree<D, E4M3, 32>(p, k, v, dk, dv, st, launches);
        case 64: return launch_tree<D, E4M3, 64>(p, k, v, dk, dv, st, launches);
        case 96: return launch_tree<D, E4M3, 96>(p, k, v, dk, dv, st, launches);
        default: return launch_tree<D, E4M3, 128>(p, k, v, dk, dv, st, launches);
    }
}

bool launch_attn_tree(TreeParams p, int D, bool e4m3, int rm, const void* K, const void* Kc, const void* Vc,
                      cudaStream_t st, int32_t* launches) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * p.cap, drows = static_cast<int64_t>(p.B) * p.Hkv * p.T;
    CUtensorMap k, v, dk, dv;
    if (!make_tmap_2d(&dk, K, drows, D, p.tp) || !make_tmap_2d(&dv, p.DV, drows, D, p.tp)) return false;
    if (e4m3) {
        if (!make_tmap_2d_u8(&k, Kc, rows, D, 64) || !make_tmap_2d_u8(&v, Vc, rows, D, 64)) return false;
        return D == 64 ? launch_tree_rows<64, true>(p, rm, k, v, dk, dv, st, launches)
                       : launch_tree_rows<128, true>(p, rm, k, v, dk, dv, st, launches);
    }
    if (!make_tmap_2d(&k, Kc, rows, D, 64) || !make_tmap_2d(&v, Vc, rows, D, 64)) return false;
    return D == 64 ? launch_tree_rows<64, false>(p, rm, k, v, dk, dv, st, launches)
                   : launch_tree_rows<128, false>(p, rm, k, v, dk, dv, st, launches);
}

}  // namespace pisa
