// Attention of a tree of drafted tokens over a K/V cache (one drafted token is plain decode).
//
//   rows   the T drafted tokens of the gh query heads that share a selection row: gh * T rows, cut
//          into row tiles of R (16 .. 96)
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
#include "pisa_tree.cuh"

namespace pisa {


// ---------------------------------------------------------------- operands

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void softmax_sync(uint32_t bar) { named_bar_sync(bar, 128); }

// N consecutive TMEM columns (16, 32 or 48) of the warp's lanes; the loads are in flight until
// tmem_wait_ld.
template <int N>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, uint32_t (&v)[N]) {
    if constexpr (N >= 32) {
        uint32_t r[32];
        tmem_ld32(taddr, r);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = r[i];
    }
    if constexpr (N % 32 == 16) {
        uint32_t r[16];
        tmem_ld16(taddr + (N - 16), r);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[N - 16 + i] = r[i];
    }
}

// ---------------------------------------------------------------- layout

template <int D, bool E4M3, int R>
struct TreeCfg {
    static constexpr int ROW = E4M3 ? D : 2 * D;         // bytes of a cache row
    static constexpr int TILE = 128 * ROW;               // K (or V) of one tile: one slot of a ring
    static constexpr int EXPS = E4M3 ? 256 : 0;          // a tile's exponent bytes of K and of V
    static constexpr int QB = R * 2 * D;                 // Q: bf16, or its two e4m3 terms
    static constexpr int PTERM = R * 128;                // one 8-bit term of P
    static constexpr int PB = E4M3 ? 3 * PTERM : 2 * PTERM;  // P: three 8-bit terms, or bf16
    // terms side by side along N (one pass over K and V for all of them) while TMEM holds them
    static constexpr bool STACK = E4M3 && R <= 64;
    static constexpr int SW = STACK ? 2 * R : R;         // TMEM columns of one S
    static constexpr int OT = STACK ? 3 : 1;             // accumulators of O
    static constexpr int COLS = 2 * SW + OT * R <= 64 ? 64 : 2 * SW + OT * R <= 128 ? 128
                                                         : 2 * SW + OT * R <= 256  ? 256
                                                                                   : 512;
    static constexpr int NWG = R >= 64 ? R / 32 : 1;     // softmax warpgroups: each takes RW columns
    static constexpr int RW = R / NWG;
    static constexpr int CW = 16;                        // columns of O taken at a time
    static constexpr int NP = !E4M3 && R > 64 ? 1 : 2;   // P buffers: one where a second would cost a slot
    static constexpr float LAZY = E4M3 ? 4.f : 8.f;      // log2 units a score may exceed the kept maximum by
    // dynamic shared memory without the rings: Q, P, masks, row parameters (8 floats a row), exponents
    static constexpr int FIXED = 1024 + QB + NP * PB + R * 8 + R * 32 + kTreeMeta * EXPS;
    static constexpr int CTAS = E4M3 && R <= 32 ? 2 : 1;  // CTAs an SM's shared memory and TMEM take
    static constexpr int THREADS = 128 * NWG + 64;
};

template <int D, bool E4M3, int R>
__global__ void __launch_bounds__(TreeCfg<D, E4M3, R>::THREADS, TreeCfg<D, E4M3, R>::CTAS)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                     const TreeParams p) {
    using C = TreeCfg<D, E4M3, R>;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* vring = ring + p.nk * C::TILE;
    uint8_t* q_s = vring + p.nv * C::TILE;
    uint8_t* p_s = q_s + C::QB;
    uint64_t* mask_s = reinterpret_cast<uint64_t*>(p_s + C::NP * C::PB);  // [R]
    float* rf_s = reinterpret_cast<float*>(mask_s + R);  // score factor of a row (e4m3: 2^-(Q's exponent))
    float* nm_s = rf_s + R;                              // -(kept maximum), 0 while there is none
    float* m_s = nm_s + R;                               // kept maximum, log2 units
    float* al_s = m_s + R;                               // factor of O and l in a rescale; 1/l at the end
    float* w_s = al_s + R;                               // [4 warps][R]
    uint8_t* exps = reinterpret_cast<uint8_t*>(w_s + 4 * R);  // [entry][K 128, V 128]
    __shared__ __align__(8) uint64_t kfull[kTreeMaxSlots], kempty[kTreeMaxSlots], vfull[kTreeMaxSlots],
        vempty[kTreeMaxSlots], sfull[2], pfull[2], pvdone[2], qfull, done;
    __shared__ int4 meta[kTreeMeta];  // kind, keys that count in the two halves
    __shared__ uint32_t tmem_slot, dflag[2], wexp[4 * C::NWG];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const TreeJob job = tree_job(p);
    if (static_cast<int64_t>(blockIdx.x) >= job.runs) return;
    int64_t pos = job.begin(blockIdx.x);
    const int64_t end = job.begin(blockIdx.x + 1);
    int64_t tile;
    int unit;
    tree_find(p, pos, tile, unit);
    if (tid == 0) {
        for (int i = 0; i < p.nk; ++i) {
            mbar_init(&kfull[i], 1);
            mbar_init(&kempty[i], 1);
        }
        for (int i = 0; i < p.nv; ++i) {
            mbar_init(&vfull[i], 1);
            mbar_init(&vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4 * C::NWG);
            mbar_init(&pvdone[i], 1);
        }
        mbar_init(&qfull, 4 * C::NWG);
        mbar_init(&done, 1);
        fence_barrier_init();
    }
    if (warp == 4 * C::NWG + 1) tmem_alloc(&tmem_slot, C::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    const uint32_t tm_o = tm + 2 * C::SW;

    bool ok = true;       // cleared by a wait that ran out: nothing more is waited for
    RingAt k, v;          // K ring (tiles and piece ends), V ring (tiles)

    if (warp == 4 * C::NWG) {
        tree_producer<D, E4M3>(p, tmK, tmV, tmDK, tmDV, ring, vring, exps, kfull, kempty, vfull, vempty, meta, pos, end,
                               tile, unit);
    } else if (warp == 4 * C::NWG + 1) {
        // ------------------------------------------------ MMA
        if (lane == 0) {
            const uint32_t q0 = smem_u32(q_s), p0 = smem_u32(p_s);
            int it = 0, pt = 0;       // S slots so far, and tiles whose P.V was issued
            int npend = 0;            // tiles whose S was issued and P.V was not (two at most: S has two buffers)
            uint32_t drafts = 0;      // bit 0: the older of them is the drafted tokens, bit 1: the younger
            uint32_t qpar = 0;
            bool issued = false;
            bool fresh = true;        // the next P.V begins O

            // K step k of P.V of the oldest pending tile
            auto pv_step = [&](int n, uint64_t a, uint64_t b) {
                if constexpr (!E4M3) {
                    mma_bf16_ss(tm_o, desc_at(a, n * 2048), desc_at(b, n * 256), idesc_bf16_f32(128, R, 1, 1),
                                !fresh || n > 0 ? 1u : 0u);
                } else if constexpr (C::STACK) {
                    mma_f8_ss(tm_o, desc_at(a, n * 32 * D), desc_at(b, n * 512), idesc_f8(3 * R, 1, 1, 1),
                              !fresh || n > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (int t = 0; t < 3; ++t)
                        mma_f8_ss(tm_o, desc_at(a, n * 32 * D), desc_at(b, t * C::PTERM + n * 512), idesc_f8(R, 1, 1, 1),
                                  !fresh || n > 0 || t > 0 ? 1u : 0u);
                }
            };
            constexpr int PVS = E4M3 ? 4 : 8, QKS = E4M3 ? D / 32 : D / 16;
            auto qk_step = [&](int n, uint32_t d, uint64_t a, uint64_t b) {
                if constexpr (!E4M3) {
                    mma_bf16_ss(d, desc_at(a, (n / 4) * 16384 + (n % 4) * 32), desc_at(b, (n / 4) * (R * 128) + (n % 4) * 32),
                                idesc_bf16_f32(128, R, 0, 0), n > 0 ? 1u : 0u);
                } else if constexpr (C::STACK) {
                    mma_f8_ss(d, desc_at(a, n * 32), desc_at(b, n * 32), idesc_f8(2 * R, 0, 0, 0), n > 0 ? 1u : 0u);
                } else {
                    mma_f8_ss(d, desc_at(a, n * 32), desc_at(b, n * 32), idesc_f8(R, 0, 0, 0), n > 0 ? 1u : 0u);
                    mma_f8_ss(d, desc_at(a, n * 32), desc_at(b, R * D + n * 32), idesc_f8(R, 1, 0, 0), 1u);
                }
            };
            auto v_desc = [&]() {
                const uint32_t vt = smem_u32(vring + v.s * C::TILE);
                if constexpr (E4M3)
                    return D == 128 ? tree_desc(vt, 0, 1024, 2) : tree_desc(vt, 0, 512, 4);
                else
                    return tree_desc(vt, D == 128 ? 16384 : 0, 1024, 2);
            };
            auto p_desc = [&]() { return tree_desc(p0 + (pt % C::NP) * C::PB, 128, 2048, 0); };
            auto p_wait = [&]() {     // P and V of the oldest pending tile are there
                ok = mbar_wait(&pfull[pt & 1], (pt >> 1) & 1, p.status, kTreeDetail | 0x05u) &&
                     mbar_wait(&vfull[v.s], v.par, p.status, kTreeDetail | 0x06u);
                tc_fence_after();
            };
            auto pv_done = [&]() {
                fresh = false;
                mma_commit(&vempty[v.s]);
                mma_commit(&pvdone[pt % C::NP]);
                v.next(p.nv);
                ++pt;
                --npend;
                drafts >>= 1;
            };
            auto pv_alone = [&]() {
                const uint64_t b = p_desc();
                if (drafts & 1u) {
                    const uint64_t a = tree_desc(smem_u32(vring + v.s * C::TILE), D == 128 ? 8192 : 0, 1024, 2);
                    for (int n = 0; n < p.tp / 16; ++n)
                        mma_bf16_ss(tm_o, desc_at(a, n * 2048), desc_at(b, n * 256), idesc_bf16_f32(128, R, 1, 1),
                                    !fresh || n > 0 ? 1u : 0u);
                } else {
                    const uint64_t a = v_desc();
#pragma unroll
                    for (int n = 0; n < PVS; ++n) pv_step(n, a, b);
                }
                pv_done();
            };
            auto flush = [&]() {
                while (npend > 0 && ok) {
                    p_wait();
                    if (ok) pv_alone();
                }
            };
            while (pos < end && ok) {
                const int b = static_cast<int>(tile / p.rows_per_seq);
                const int units = tree_units(p, tree_len(p, b));
                const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
                ok = mbar_wait(&qfull, qpar, p.status, kTreeDetail | 0x07u);
                qpar ^= 1u;
                fresh = true;
                while (ok) {
                    // the next S goes where the older pending tile's was: its P.V comes first, or, if the next
                    // K is there, step by step with it (two chains of dependent products side by side)
                    bool both = false;
                    if (npend == 2) {
                        p_wait();
                        if (!ok) break;
                        both = (drafts & 1u) == 0 && mbar_test(&kfull[k.s], k.par);
                        if (!both) pv_alone();
                    }
                    ok = mbar_wait(&kfull[k.s], k.par, p.status, kTreeDetail | 0x08u);
                    if (!ok) break;
                    const int kind = meta[k.n % kTreeMeta].x;
                    if (both && kind != kTileCache) {
                        pv_alone();
                        both = false;
                    }
                    issued = true;
                    if (kind == kTileEnd) {
                        flush();
                        if (ok) {
                            // with every product of the piece complete, the softmax may read O
                            mma_commit(&sfull[it & 1]);
                            mbar_arrive(&kempty[k.s]);
                            ++it;
                            k.next(p.nk);
                        }
                        break;
                    }
                    if (E4M3 && kind == kTileDraft) {
                        // Q comes again, as bf16: a slot without scores tells the softmax so
                        flush();
                        if (!ok) break;
                        mma_commit(&sfull[it & 1]);
                        ++it;
                        ok = mbar_wait(&qfull, qpar, p.status, kTreeDetail | 0x09u);
                        qpar ^= 1u;
                        if (!ok) break;
                    }
                    tc_fence_after();
                    const uint32_t kt = smem_u32(ring + k.s * C::TILE);
                    const uint32_t d = tm + (it & 1) * C::SW;
                    if (kind == kTileDraft) {
                        const uint64_t a = tree_desc(kt, 16, 1024, 2), bq = tree_desc(q0, 16, 1024, 2);
#pragma unroll
                        for (int n = 0; n < D / 16; ++n)
                            mma_bf16_ss(d, desc_at(a, (n / 4) * 8192 + (n % 4) * 32), desc_at(bq, (n / 4) * (R * 128) + (n % 4) * 32),
                                        idesc_bf16_f32(128, R, 0, 0), n > 0 ? 1u : 0u);
                    } else {
                        const uint64_t a = E4M3 && D == 64 ? tree_desc(kt, 16, 512, 4) : tree_desc(kt, 16, 1024, 2);
                        const uint64_t bq = E4M3 && D == 64 ? tree_desc(q0, 16, 512, 4) : tree_desc(q0, 16, 1024, 2);
                        const uint64_t va = v_desc(), pb = p_desc();
#pragma unroll
                        for (int n = 0; n < PVS; ++n) {
                            if (both) pv_step(n, va, pb);
                            if (n < QKS) qk_step(n, d, a, bq);
                        }
                    }
                    mma_commit(&sfull[it & 1]);
                    mma_commit(&kempty[k.s]);
                    if (both) pv_done();
                    if (kind == kTileDraft) drafts |= 1u << npend;
                    ++npend;
                    ++it;
                    k.next(p.nk);
                }
                pos += u1 - unit;
                unit = 0;
                ++tile;
            }
            if (issued) {  // nothing of this CTA's still runs when TMEM goes
                mma_commit(&done);
                mbar_wait(&done, 0, p.status, kTreeDetail | 0x0Au);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax: thread = key of the tile = TMEM lane
        // With two warpgroups each takes RW of the rows, on its own: its maxima, its unit, its columns of
        // O, its barrier.
        const int wg = warp / 4, key = tid & 127, cb = wg * C::RW;
        const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;  // TMEM lane base of the warp
        const uint32_t bar = 1 + wg;
        const int rows = p.gh * p.T;
        float *rf = rf_s + cb, *nms = nm_s + cb, *ms = m_s + cb, *als = al_s + cb, *ws = w_s + 4 * cb;
        const uint64_t* masks = mask_s + cb;
        int it = 0, pt = 0;
        while (pos < end && ok) {
            const int b = static_cast<int>(tile / p.rows_per_seq);
            const int rem = static_cast<int>(tile % p.rows_per_seq);
            const int hs = rem / p.mt, row_base = (rem % p.mt) * R + cb;
            const int units = tree_units(p, tree_len(p, b));
            const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
            const int64_t out0 = (static_cast<int64_t>(b) * p.Hq + hs * p.gh) * p.T;  // first row of the group
            const int nrows = max(0, min(C::RW, rows - row_base));
            const uint4* qg = reinterpret_cast<const uint4*>(p.Q + (out0 + row_base) * D);

            // Q as bf16: [D / 64][R rows][128 B], 128-byte swizzle
            auto q_bf16 = [&]() {
                for (int e = key; e < C::RW * (D / 8); e += 128) {
                    const int r = e / (D / 8) + cb, c = e % (D / 8);
                    const uint4 x = r - cb < nrows ? __ldg(qg + e) : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(q_s + (c / 8) * (R * 128) + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = x;
                }
            };
            // Q as two 8-bit terms [R rows][D B], swizzled by the row's size; D/8 lanes hold a row
            auto q_terms = [&]() {
                for (int e = key; e < C::RW * (D / 8); e += 128) {  // RW * D / 8 is a multiple of 128
                    const int r = e / (D / 8) + cb, c = e % (D / 8);
                    const uint4 x = r - cb < nrows ? __ldg(qg + e) : make_uint4(0u, 0u, 0u, 0u);
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
                        // the remainder; stacked terms have sums of their own, so it can be kept 16 times larger
                        lo[k] = C::STACK ? cvt_e4m3x2((a - h.x) * 16.f, (bb - h.y) * 16.f) : cvt_e5m2x2(a - h.x, bb - h.y);
                        // an infinity saturates the first term: the second makes the score a NaN
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
            if (u1 == units && key < C::RW) {  // this piece ends with the drafted tokens
                const int rg = row_base + key;
                const uint64_t live = p.T == 64 ? ~0ull : (1ull << p.T) - 1ull;
                mask_s[cb + key] = rg < rows ? __ldg(p.mask + static_cast<int64_t>(b) * p.T + rg % p.T) & live : 0ull;
            }
            // Q of this piece may be announced: the MMA lane saw the piece before to its end (the slot that
            // ends a piece comes through it)
            q_ready();
            if (key < C::RW) nms[key] = 0.f;
            softmax_sync(bar);  // row factors and masks

            uint64_t l2[C::RW / 2];  // this key's share of the rows' sums
#pragma unroll
            for (int i = 0; i < C::RW / 2; ++i) l2[i] = 0ull;
            // bf16: the kept maxima in registers (a shared-memory load waits for the products' operand reads)
            uint64_t nm2[E4M3 ? 1 : C::RW / 2];
            if constexpr (!E4M3) {
#pragma unroll
                for (int i = 0; i < C::RW / 2; ++i) nm2[i] = 0ull;
            }
            bool fresh = true, cached = false;  // no tile yet; a tile of the cache so far
            int u = 0, uexp = 0;   // unit exponent of O, and the V exponent it was set by (e4m3)

            while (true) {
                // Every slot is one barrier, and a second one when the first says so: a warp whose wait ran
                // out takes both, so that all warps leave together whatever the others saw in the slot.
                if (ok) ok = mbar_wait(&sfull[it & 1], (it >> 1) & 1, p.status, kTreeDetail | 0x0Bu);
                ok = __all_sync(0xFFFFFFFFu, ok);
                tc_fence_after();
                const int me = k.n % kTreeMeta;
                const int4 mt = ok ? meta[me] : make_int4(kTileEnd, 0, 0, 0);
                if (E4M3 && mt.x == kTileDraft) {
                    // this slot only says that the drafted tokens come: every S so far is formed, Q's buffer
                    // is free for the bf16 rows; the next slot has the scores
                    q_bf16();
                    q_ready();
                    ++it;
                    ok = mbar_wait(&sfull[it & 1], (it >> 1) & 1, p.status, kTreeDetail | 0x0Cu);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    tc_fence_after();
                }
                if (mt.x == kTileEnd) {
                    if (vote_any(bar, 128, !ok) && vote_any(bar, 128, !ok)) ok = false;
                    ++it;
                    k.next(p.nk);
                    break;
                }
                const bool draft = mt.x == kTileDraft;
                uint8_t* vt = vring + v.s * C::TILE;
                const bool valid = draft ? key < p.T : (key & 63) < (key < 64 ? mt.y : mt.z);
                const bool partial = draft || mt.y < 64 || mt.z < 64;
                float kf = p.scale_log2;
                int ev = 0;
                if (E4M3 && !draft && valid) {
                    kf *= __uint_as_float(static_cast<uint32_t>(exps[me * 256 + key]) << 23);
                    ev = exps[me * 256 + 128 + key];
                }
                if (draft && wg == 0 && key < 2) dflag[key] = 0;
                // scores against the kept maximum, log2 units: x = acc * kf (* the row's factor) - m
                const uint32_t ts = tm + lanes + (it & 1) * C::SW + cb;
                uint64_t x[C::RW / 2];
                {
                    uint32_t v[C::RW];
                    tmem_cols<C::RW>(ts, v);
                    if (C::STACK && !draft) {  // the second term of Q is 16 times too large
                        uint32_t w[C::RW];
                        tmem_cols<C::RW>(ts + R, w);
                        tmem_wait_ld();
                        const uint64_t f = f2_pack(0.0625f, 0.0625f);
#pragma unroll
                        for (int i = 0; i < C::RW / 2; ++i)
                            x[i] = f2_fma(f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), f,
                                          f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])));
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < C::RW / 2; ++i)
                            x[i] = f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    }
                }
                const uint64_t kf2 = f2_pack(kf, kf);
#pragma unroll
                for (int i = 0; i < C::RW / 4; ++i) {
                    if constexpr (E4M3) {
                        const float4 nm = *reinterpret_cast<const float4*>(nms + 4 * i);
                        float4 f = *reinterpret_cast<const float4*>(rf + 4 * i);
                        if (draft) f = make_float4(1.f, 1.f, 1.f, 1.f);  // bf16 rows as they are
                        x[2 * i] = f2_fma(f2_mul(x[2 * i], kf2), f2_pack(f.x, f.y), f2_pack(nm.x, nm.y));
                        x[2 * i + 1] = f2_fma(f2_mul(x[2 * i + 1], kf2), f2_pack(f.z, f.w), f2_pack(nm.z, nm.w));
                    } else {
                        x[2 * i] = f2_fma(x[2 * i], kf2, nm2[2 * i]);
                        x[2 * i + 1] = f2_fma(x[2 * i + 1], kf2, nm2[2 * i + 1]);
                    }
                }
                if (partial) {
                    const uint64_t none = f2_pack(-INFINITY, -INFINITY);
                    if (draft) {
#pragma unroll
                        for (int i = 0; i < C::RW / 2; ++i) {
                            float lo, hi;
                            f2_unpack(x[i], lo, hi);
                            lo = valid && (masks[2 * i] >> key) & 1ull ? lo : -INFINITY;
                            hi = valid && (masks[2 * i + 1] >> key) & 1ull ? hi : -INFINITY;
                            x[i] = f2_pack(lo, hi);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < C::RW / 2; ++i) x[i] = valid ? x[i] : none;
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < C::RW / 2; ++i) {
                    float lo, hi;
                    f2_unpack(x[i], lo, hi);
                    top = fmax3(top, lo, hi);
                }
                const bool over = top > C::LAZY || (E4M3 && ev > uexp);
                if (vote_any(bar, 128, !ok || fresh || over)) {
                    if (vote_any(bar, 128, !ok)) {
                        ok = false;
                        break;
                    }
                    // the rows' maxima over this tile (less the kept ones), and the largest V exponent
                    float mine = -INFINITY;
#pragma unroll
                    for (int i = 0; i < C::RW / 2; ++i) {
                        float lo, hi;
                        f2_unpack(x[i], lo, hi);
                        lo = warp_max(lo);
                        hi = warp_max(hi);
                        if (lane == (2 * i) % 32) mine = lo;
                        if (lane == (2 * i) % 32 + 1) mine = hi;
                        if (2 * i + 2 == C::RW || (2 * i + 2) % 32 == 0) {
                            const int c = (2 * i) / 32 * 32 + lane;
                            if (c < C::RW) ws[(warp % 4) * C::RW + c] = mine;
                        }
                    }
                    if constexpr (E4M3) {
                        const uint32_t we = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(ev));
                        if (lane == 0) wexp[warp] = we;
                    }
                    softmax_sync(bar);
                    if (key < C::RW) {
                        const float M = fmaxf(fmaxf(ws[key], ws[C::RW + key]), fmaxf(ws[2 * C::RW + key], ws[3 * C::RW + key]));
                        const float was = -nms[key];  // the reference that x was taken against
                        const float old = fresh ? -INFINITY : ms[key];
                        const float now = fmaxf(old, was + M);
                        als[key] = now == old ? 1.f : fast_exp2(old - now);
                        ms[key] = now;
                        nms[key] = now == -INFINITY ? 0.f : -now;
                        ws[key] = was + nms[key];     // what brings x to the new reference
                    }
                    float uf = 1.f;
                    if (E4M3 && !draft) {
                        const uint32_t* we = wexp + 4 * wg;
                        const int e = static_cast<int>(min(254u, max(max(we[0], we[1]), max(we[2], we[3]))));
                        if (fresh || e > uexp) {
                            uexp = e;
                            const int un = max(kTreeUMin, e - 127 + static_cast<int>(C::LAZY) - 15);
                            uf = pow2i(max(-126, u - un));  // u - un <= 0 once O holds anything
                            u = un;
                        }
                    }
                    softmax_sync(bar);
#pragma unroll
                    for (int i = 0; i < C::RW / 4; ++i) {
                        const float4 d = *reinterpret_cast<const float4*>(ws + 4 * i);
                        x[2 * i] = f2_add(x[2 * i], f2_pack(d.x, d.y));
                        x[2 * i + 1] = f2_add(x[2 * i + 1], f2_pack(d.z, d.w));
                        if constexpr (!E4M3) {
                            const float4 nm = *reinterpret_cast<const float4*>(nms + 4 * i);
                            nm2[2 * i] = f2_pack(nm.x, nm.y);
                            nm2[2 * i + 1] = f2_pack(nm.z, nm.w);
                        }
                    }
                    if (!fresh) {
                        const int j = pt - 1;
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pvdone[j % C::NP], (j / C::NP) & 1, p.status,
                                                               kTreeDetail | 0x0Du));
                        tc_fence_after();
#pragma unroll 1
                        for (int t = 0; t < (cached ? C::OT : 1); ++t) {
#pragma unroll 1
                            for (int c0 = 0; c0 < C::RW; c0 += C::CW) {
                                const uint32_t to = tm_o + lanes + t * R + cb + c0;
                                uint32_t v[C::CW];
                                tmem_ld16(to, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < C::CW; ++i)
                                    v[i] = __float_as_uint(__uint_as_float(v[i]) * (als[c0 + i] * uf));
                                tmem_st16(to, v);
                            }
                        }
                        tmem_wait_st();
#pragma unroll
                        for (int i = 0; i < C::RW / 4; ++i) {
                            const float4 a = *reinterpret_cast<const float4*>(als + 4 * i);
                            l2[2 * i] = f2_mul(l2[2 * i], f2_pack(a.x, a.y));
                            l2[2 * i + 1] = f2_mul(l2[2 * i + 1], f2_pack(a.z, a.w));
                        }
                    }
                    fresh = false;
                }
                // With two buffers P's is free: this tile's S is complete, and with it every product issued
                // before it, the P.V of two tiles before among them.
                uint8_t* pb = p_s + (pt % C::NP) * C::PB;
#pragma unroll
                for (int i = 0; i < C::RW / 2; ++i) {
                    float lo, hi;
                    f2_unpack(x[i], lo, hi);
                    x[i] = f2_pack(fast_exp2(lo), fast_exp2(hi));
                    l2[i] = f2_add(l2[i], x[i]);
                }
                if (C::NP == 1 && pt > 0 && ok)  // the one buffer: the last P.V has read it
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pvdone[0], (pt - 1) & 1, p.status, kTreeDetail | 0x0Eu));
                if constexpr (E4M3) {
                    // a row of exponent 255 stands for NaN (its bytes are zero); a row that does not count has
                    // P = 0 and a factor of 2^-126
                    const float pf = draft ? pow2i(min(127, max(-126, -u)))
                                           : __uint_as_float(ev == 255 ? 0x7FFFFFFFu : static_cast<uint32_t>(max(ev - u, 1)) << 23);
                    const uint64_t pf2 = f2_pack(pf, pf);
#pragma unroll
                    for (int i = 0; i < C::RW / 2; ++i) x[i] = f2_mul(x[i], pf2);
                }
                if (E4M3 && !draft) {
#pragma unroll
                    for (int g = 0; g < C::RW / 16; ++g) {
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
                        uint8_t* dst = pb + (cb / 16 + g) * 2048 + key * 16;
                        *reinterpret_cast<uint4*>(dst) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                        *reinterpret_cast<uint4*>(dst + C::PTERM) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
                        *reinterpret_cast<uint4*>(dst + 2 * C::PTERM) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < C::RW / 8; ++g) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float lo, hi;
                            f2_unpack(x[4 * g + k], lo, hi);
                            w[k] = pack_bf16x2(lo, hi);
                        }
                        *reinterpret_cast<uint4*>(pb + (cb / 8 + g) * 2048 + key * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (wg == 0 && partial && ok)  // what follows writes V's tile: it has landed
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&vfull[v.s], v.par, p.status, kTreeDetail | 0x0Fu));
                if (wg == 0 && partial && !valid && !draft) {
                    // what the cache holds past the sequence must not meet P's zeros as a NaN
                    for (int c = 0; c < C::ROW / 16; ++c) {
                        uint8_t* z = vt + (E4M3 ? key * D + 16 * c : (c / 8) * 16384 + key * 128 + 16 * (c % 8));
                        *reinterpret_cast<uint4*>(z) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                if (wg == 0 && draft && key < p.tp) {
                    // a drafted value that is not finite would reach every token through 0 * x: it is taken
                    // out here and given to the tokens that attend it at the end
                    uint32_t bad = 0;
                    for (int c = 0; c < D / 8; ++c) {
                        uint4* z = reinterpret_cast<uint4*>(vt + (c / 8) * 8192 + key * 128 + 16 * (c % 8));
                        uint32_t w[4] = {z->x, z->y, z->z, z->w};
                        uint32_t any = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((w[k] & 0x7F80u) == 0x7F80u) w[k] &= 0xFFFF0000u, any = 1;
                            if ((w[k] & 0x7F800000u) == 0x7F800000u) w[k] &= 0x0000FFFFu, any = 1;
                        }
                        if (!valid) {
                            *z = make_uint4(0u, 0u, 0u, 0u);
                        } else if (any) {
                            *z = make_uint4(w[0], w[1], w[2], w[3]);
                            bad = 1;
                        }
                    }
                    if (bad) atomicOr(&dflag[key >> 5], 1u << (key & 31));
                }
                cached = cached || !draft;
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[pt & 1]);
                ++it;
                ++pt;
                k.next(p.nk);
                v.next(p.nv);
            }
            if (!ok) break;

            // ---- the piece's end (every product is complete): sums over the keys, then O^T (lane = dim) to
            // its rows
            const bool any_tile = !fresh;
#pragma unroll
            for (int c0 = 0; c0 < C::RW; c0 += 16) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) f2_unpack(l2[c0 / 2 + i], v[2 * i], v[2 * i + 1]);
                // lanes j and j + 16 end with the sum of column j: halves are exchanged, the kept half is added
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 16);
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
                if (lane < 16) ws[(warp % 4) * C::RW + c0 + lane] = v[0];
            }
            softmax_sync(bar);
            const bool whole = unit == 0 && u1 == units;
            // partial slots: 2c for a piece that goes on with a row tile, 2c + 1 for one that begins it
            float* part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (unit == 0 ? 1 : 0)) * R * (D + 2);
            if (key < C::RW) {
                const float l = (ws[key] + ws[C::RW + key]) + (ws[2 * C::RW + key] + ws[3 * C::RW + key]);
                const float m = any_tile ? ms[key] : -INFINITY;
                als[key] = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                if (whole) {
                    if (p.lse != nullptr && key < nrows)
                        p.lse[out0 + row_base + key] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                } else {
                    part[R * D + 2 * (cb + key)] = l == 0.f ? -INFINITY : m;
                    part[R * D + 2 * (cb + key) + 1] = l;
                }
            }
            softmax_sync(bar);
            const float uf = E4M3 ? pow2i(min(127, max(-126, u))) : 1.f;
            const uint64_t odd = u1 == units ? dflag[0] | (static_cast<uint64_t>(dflag[1]) << 32) : 0ull;
            const int kvh = p.per_qhead ? hs / p.g : hs;
#pragma unroll 1
            for (int c0 = 0; c0 < C::RW; c0 += C::CW) {
                if (c0 >= nrows) break;
                uint32_t v[C::CW];
                if (any_tile) {
                    tmem_ld16(tm_o + lanes + cb + c0, v);
                    tmem_wait_ld();
                    if (C::OT > 1 && cached) {
#pragma unroll
                        for (int t = 1; t < C::OT; ++t) {
                            uint32_t w[C::CW];
                            tmem_ld16(tm_o + lanes + t * R + cb + c0, w);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < C::CW; ++i)
                                v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < C::CW; ++i) v[i] = 0u;
                }
                if (key < D) {
#pragma unroll
                    for (int i = 0; i < C::CW; ++i) {
                        const int r = c0 + i;
                        if (r < nrows) {
                            float o = __uint_as_float(v[i]) * (uf * als[r]);
                            if (odd != 0) {
                                for (uint64_t left = odd & masks[r]; left != 0; left &= left - 1) {
                                    const int jd = __ffsll(static_cast<long long>(left)) - 1;
                                    const float y = __bfloat162float(
                                        p.DV[((static_cast<int64_t>(b) * p.Hkv + kvh) * p.T + jd) * D + key]);
                                    if (!isfinite(y)) o += y;
                                }
                            }
                            if (whole)
                                p.O[(out0 + row_base + r) * D + key] = __float2bfloat16_rn(o);
                            else
                                part[(cb + r) * D + key] = o;
                        }
                    }
                }
            }
            tc_fence_before();
            softmax_sync(bar);  // row parameters are free for the next piece
            pos += u1 - unit;
            unit = 0;
            ++tile;
        }
    }
    __syncthreads();
    if (warp == 4 * C::NWG + 1) {
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
    const int hs = rem / p.mt, row_base = (rem % p.mt) * p.rpt;
    const int rows = p.gh * p.T;
    const int row = static_cast<int>(blockIdx.y) * 4 + static_cast<int>(threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row >= p.rpt || row_base + row >= rows) return;
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

// Rows of one row tile for a selection row of `rows` rows: 8 or 16 (attn_tree_few.cu), 32 (here), 128 or
// 256 (attn_tree_many.cu); past 256 rows several tiles share them evenly.
int tree_row_tile(int rows) {
    for (int r : {8, 16, 32, 128})
        if (rows <= r) return r;
    return 256;
}

// CTAs on one SM: as many as its shared memory takes.
int tree_ctas_per_sm(int rm, bool e4m3) { return e4m3 && rm == 8 ? 3 : rm <= 16 || (e4m3 && rm <= 32) ? 2 : 1; }

bool launch_tree_merge(const TreeParams& p, int D, int rm, cudaStream_t st, int32_t* launches) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.rows_per_seq, rm / 4);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = D == 64 ? cudaLaunchKernelEx(&cfg, attn_tree_merge_kernel<64>, p, rm)
                                  : cudaLaunchKernelEx(&cfg, attn_tree_merge_kernel<128>, p, rm);
    if (e != cudaSuccess) return false;
    ++*launches;
    return true;
}

template <int D, bool E4M3, int R>
static bool launch_tree(TreeParams p, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dk,
                        const CUtensorMap& dv, cudaStream_t st, int32_t* launches) {
    using C = TreeCfg<D, E4M3, R>;
    constexpr int budget = (C::CTAS == 2 ? 112 : 225) * 1024;
    constexpr int fit = (budget - C::FIXED) / C::TILE;
    constexpr int slots = fit < 2 * kTreeMaxSlots ? fit : 2 * kTreeMaxSlots;
    static_assert(slots >= 4, "two slots of K and of V must fit");
    p.nk = slots / 2;
    p.nv = slots - p.nk;
    const int smem = C::FIXED + slots * C::TILE;
    static std::atomic<uint64_t> configured{0};
    if (!configure_smem_once(reinterpret_cast<const void*>(attn_tree_kernel<D, E4M3, R>), smem, configured)) return false;
    attn_tree_kernel<D, E4M3, R><<<p.runs, C::THREADS, smem, st>>>(k, v, dk, dv, p);
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    return launch_tree_merge(p, D, R, st, launches);
}

template <int D, bool E4M3>
static bool launch_tree_rows(const TreeParams& p, int rm, const CUtensorMap& k, const CUtensorMap& v,
                             const CUtensorMap& dk, const CUtensorMap& dv, cudaStream_t st, int32_t* launches) {
    switch (rm) {
        case 32: return launch_tree<D, E4M3, 32>(p, k, v, dk, dv, st, launches);
        case 64: return launch_tree<D, E4M3, 64>(p, k, v, dk, dv, st, launches);
        default: return launch_tree<D, E4M3, 96>(p, k, v, dk, dv, st, launches);
    }
}

bool launch_attn_tree(TreeParams p, int D, bool e4m3, int rm, const void* K, const void* Kc, const void* Vc,
                      cudaStream_t st, int32_t* launches) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * p.cap, drows = static_cast<int64_t>(p.B) * p.Hkv * p.T;
    CUtensorMap k, v, dk, dv;
    if (rm <= 16) return launch_attn_tree_few(p, D, e4m3, rm, K, Kc, Vc, st, launches);
    if (rm >= 128) return launch_attn_tree_many(p, D, e4m3, rm, K, Kc, Vc, st, launches);
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
