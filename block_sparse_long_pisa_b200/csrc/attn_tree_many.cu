// Tree attention for many rows: more than 32 drafted-token-and-head rows per selection row. The function,
// the cut into runs and the treatment of the drafted tokens are those of attn_tree.cu; here the tensor
// cores and the exponentials count as much as the bytes.
//
// Rows on the M side, 128 to a tile, one or two tiles in a CTA: S = Q K^T and O = P V with P read from
// TMEM, so a score costs no shared memory at all (with the keys on the M side, attn_tree.cu, K and V are
// fetched as the 128-lane operand for every 96 rows, the values transposed at half the rate, and P goes
// through shared memory: 363 us for trees of 48 tokens of four heads over 8 ragged bf16 caches). A
// row belongs to two softmax threads, one for each half of a tile's keys (one thread for all of them made the
// softmax the longer side of every tile: 314 us); the two warps meet in one vote a tile.
//
// A tile is 128 keys (two units of the cache, or the drafted tokens). Two passes over S in TMEM: the row's
// maximum (the kept one moves when a score exceeds it by 2^LAZY, and O with it, by the two warps), then
// the probabilities, written as operand A of P V over the columns of S that have been read. Order of the
// MMA lane with two row tiles: S(0, g), P V(1, g - 1), S(1, g), P V(0, g): the softmax of one runs under the
// products of the other; with one row tile S has two buffers and the order is S(g), P V(g - 1).
//
// e4m3: Q as e4m3 + e5m2 terms, P as three e5m2 terms, exponents as in attn_tree.cu; the key's two exponent
// factors come from a table that the warps of a row tile fill for each tile of keys.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pisa_device.cuh"
#include "pisa_tree.cuh"

namespace pisa {

template <int D, bool E4M3, int NM>
struct ManyCfg {
    static constexpr int ROW = E4M3 ? D : 2 * D;
    static constexpr int TILE = 128 * ROW;               // one slot of a ring
    static constexpr int EXPS = E4M3 ? 256 : 0;
    static constexpr int QB = 128 * 2 * D;               // one row tile of Q: bf16, or its two 8-bit terms
    static constexpr int FACT = E4M3 ? 1024 : 0;         // factors of 128 keys: K's, then V's
    static constexpr int FIXED = 1024 + NM * (QB + FACT + 1024) + kTreeMeta * EXPS;  // 1024: [half][row] exchange
    static constexpr int RM = 128 * NM;
    static constexpr int THREADS = 256 * NM + 64;
    static constexpr int O_COL = 256;                    // S: two of 128 columns (row tiles, or buffers)
    static constexpr float LAZY = E4M3 ? 4.f : 8.f;      // log2 units a score may exceed the kept maximum by
};

// D[tmem] (+)= A[tmem] * B[smem]: 8-bit A, four values to a column.
__device__ __forceinline__ void mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// kind::f8f6f4, A e4m3 (0) or e5m2 (1), B e4m3, M = 128
__host__ __device__ constexpr uint32_t idesc_f8_a(int n, int a_type, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(a_type) << 7) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

template <int D, bool E4M3, int NM>
__global__ void __launch_bounds__(ManyCfg<D, E4M3, NM>::THREADS, 1)
    attn_tree_many_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                          const TreeParams p) {
    using C = ManyCfg<D, E4M3, NM>;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* vring = ring + p.nk * C::TILE;
    uint8_t* q_s = vring + p.nv * C::TILE;               // [row tile][QB]
    float* fact = reinterpret_cast<float*>(q_s + NM * C::QB);          // [row tile][K 128, V 128]
    float* xch = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(fact) + NM * C::FACT);  // [row tile][half][128]
    uint8_t* exps = reinterpret_cast<uint8_t*>(xch) + NM * 1024;       // [entry][K 128, V 128]
    __shared__ __align__(8) uint64_t kfull[kTreeMaxSlots], kempty[kTreeMaxSlots], vfull[kTreeMaxSlots],
        vempty[kTreeMaxSlots], sfull[2], pfull[2], pvdone[2], qfull, done;
    __shared__ int4 meta[kTreeMeta];  // kind, keys that count in the two halves
    __shared__ uint32_t tmem_slot, dflag[2][2];

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
            mbar_init(&pfull[i], 8);
            mbar_init(&pvdone[i], 1);
            dflag[0][i] = dflag[1][i] = 0;
        }
        mbar_init(&qfull, 8 * NM);
        mbar_init(&done, 1);
        fence_barrier_init();
    }
    if (warp == 8 * NM + 1) tmem_alloc(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    bool ok = true;       // cleared by a wait that ran out: nothing more is waited for
    RingAt k, v;          // K ring (tiles and piece ends), V ring (tiles)
    // Row tile h and number n of a tile (or of an S slot) -> barrier, its parity, and the columns of S.
    auto bar_of = [](int h, int n) { return NM == 2 ? h : n & 1; };
    auto par_of = [](int n) { return static_cast<uint32_t>((NM == 2 ? n : n >> 1) & 1); };

    if (warp == 8 * NM) {
        tree_producer<D, E4M3>(p, tmK, tmV, tmDK, tmDV, ring, vring, exps, kfull, kempty, vfull, vempty, meta, pos, end,
                               tile, unit);
    } else if (warp == 8 * NM + 1) {
        // ------------------------------------------------ MMA
        if (lane == 0) {
            const uint32_t q0 = smem_u32(q_s);
            int it = 0, tn = 0;       // S slots so far, and tiles among them
            int pn = 0, pit = 0;      // tiles whose P V was issued for every row tile; the S slot of the next one
            bool pend = false;        // P V of the tile before is still to be issued (two row tiles: for tile 1)
            bool pdraft = false;      // and that tile is the drafted tokens
            bool fresh[2] = {true, true};  // the next P V begins O
            uint32_t qpar = 0;
            bool issued = false;
            // S of row tile h from the K slot at hand
            auto qk = [&](int h, bool draft) {
                const uint32_t kt = smem_u32(ring + k.s * C::TILE), qt = q0 + h * C::QB;
                const uint32_t d = tm + bar_of(h, it) * 128;
                if (draft || !E4M3) {
                    const uint32_t sub = draft ? 8192 : 16384;
                    const uint64_t a = tree_desc(qt, 16, 1024, 2), b = tree_desc(kt, 16, 1024, 2);
                    const uint32_t id = idesc_bf16_f32(128, draft ? p.tp : 128, 0, 0);
#pragma unroll
                    for (int n = 0; n < D / 16; ++n)
                        mma_bf16_ss(d, desc_at(a, (n / 4) * 16384 + (n % 4) * 32), desc_at(b, (n / 4) * sub + (n % 4) * 32), id,
                                    n > 0 ? 1u : 0u);
                } else {
                    const uint64_t a = D == 128 ? tree_desc(qt, 16, 1024, 2) : tree_desc(qt, 16, 512, 4);
                    const uint64_t b = D == 128 ? tree_desc(kt, 16, 1024, 2) : tree_desc(kt, 16, 512, 4);
#pragma unroll
                    for (int n = 0; n < D / 32; ++n) {
                        mma_f8_ss(d, desc_at(a, n * 32), desc_at(b, n * 32), idesc_f8_a(128, 0, 0), n > 0 ? 1u : 0u);
                        mma_f8_ss(d, desc_at(a, 128 * D + n * 32), desc_at(b, n * 32), idesc_f8_a(128, 1, 0), 1u);
                    }
                }
                mma_commit(&sfull[bar_of(h, it)]);
            };
            // P V of row tile h for tile number n (S slot sit) from the V slot at hand
            auto pv = [&](int h, int n, int sit, bool draft) {
                ok = mbar_wait(&pfull[bar_of(h, n)], par_of(n), p.status, kTreeDetail | 0x21u) &&
                     mbar_wait(&vfull[v.s], v.par, p.status, kTreeDetail | 0x22u);
                if (!ok) return;
                tc_fence_after();
                const uint32_t vt = smem_u32(vring + v.s * C::TILE);
                const uint32_t a = tm + bar_of(h, sit) * 128, d = tm + C::O_COL + h * 128;
                if (draft || !E4M3) {
                    const uint64_t b = tree_desc(vt, draft ? 8192 : 16384, 1024, 2);
                    const int steps = draft ? p.tp / 16 : 8;
                    for (int i = 0; i < steps; ++i)
                        mma_bf16_ts(d, a + 32 * (i / 2) + 8 * (i % 2), desc_at(b, i * 2048), idesc_bf16_f32(128, D, 0, 1),
                                    !fresh[h] || i > 0 ? 1u : 0u);
                } else {
                    const uint64_t b = D == 128 ? tree_desc(vt, 0, 1024, 2) : tree_desc(vt, 0, 512, 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int t = 0; t < 3; ++t)
                            mma_f8_ts(d, a + 32 * i + 8 * t, desc_at(b, i * 32 * D), idesc_f8_a(D, 1, 1),
                                      !fresh[h] || i > 0 || t > 0 ? 1u : 0u);
                    }
                }
                fresh[h] = false;
                mma_commit(&pvdone[bar_of(h, n)]);
            };
            // the P V that is still to be issued (two row tiles: of tile 1), and with it the V slot's release
            auto flush = [&]() {
                if (!pend || !ok) return;
                pv(NM - 1, pn, pit, pdraft);
                if (!ok) return;
                mma_commit(&vempty[v.s]);
                v.next(p.nv);
                ++pn;
                pend = false;
            };
            auto announce = [&]() {  // an S slot without scores, after every product so far
                issued = true;
                mma_commit(&sfull[bar_of(0, it)]);
                if (NM == 2) mma_commit(&sfull[1]);
                ++it;
            };
            while (pos < end && ok) {
                const int b = static_cast<int>(tile / p.rows_per_seq);
                const int units = tree_units(p, tree_len(p, b));
                const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
                ok = mbar_wait(&qfull, qpar, p.status, kTreeDetail | 0x23u);
                qpar ^= 1u;
                fresh[0] = fresh[1] = true;
                while (ok) {
                    ok = mbar_wait(&kfull[k.s], k.par, p.status, kTreeDetail | 0x24u);
                    if (!ok) break;
                    const int kind = meta[k.n % kTreeMeta].x;
                    const bool draft = kind == kTileDraft;
                    if (kind == kTileEnd) {
                        flush();
                        if (ok) {
                            announce();  // the softmax may read O
                            mbar_arrive(&kempty[k.s]);
                            k.next(p.nk);
                        }
                        break;
                    }
                    if (E4M3 && draft) {  // Q comes again, as bf16
                        flush();
                        if (!ok) break;
                        announce();
                        ok = mbar_wait(&qfull, qpar, p.status, kTreeDetail | 0x25u);
                        qpar ^= 1u;
                        if (!ok) break;
                    }
                    // S goes where an earlier tile's P is read from: two row tiles, the tile before's; one row
                    // tile, that of two before
                    const int back = NM == 2 ? 1 : 2;
                    auto free_s = [&](int h) {
                        if (tn >= back)
                            ok = mbar_wait(&pvdone[bar_of(h, tn - back)], par_of(tn - back), p.status, kTreeDetail | 0x26u);
                        tc_fence_after();
                        return ok;
                    };
                    issued = true;
                    if (!free_s(0)) break;
                    qk(0, draft);
                    if constexpr (NM == 2) {
                        flush();          // P V(1) of the tile before
                        if (!ok || !free_s(1)) break;
                        qk(1, draft);
                        mma_commit(&kempty[k.s]);
                        pv(0, tn, it, draft);
                        if (!ok) break;
                    } else {
                        mma_commit(&kempty[k.s]);
                        flush();
                        if (!ok) break;
                    }
                    pend = true;
                    pdraft = draft;
                    pit = it;
                    ++tn;
                    ++it;
                    k.next(p.nk);
                }
                pos += u1 - unit;
                unit = 0;
                ++tile;
            }
            if (issued) {  // nothing of this CTA's still runs when TMEM goes
                mma_commit(&done);
                mbar_wait(&done, 0, p.status, kTreeDetail | 0x27u);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax: a row of row tile h (TMEM lane), half of
        // a tile's keys
        const int h = (warp / 4) % NM, half = warp / (4 * NM), row = tid & 127;
        const uint32_t pair = 1 + 4 * h + warp % 4, group = 9 + h;  // barriers of the row's two warps, of the row tile
        float* mine_x = xch + h * 256 + half * 128 + row;
        const float* other_x = xch + h * 256 + (1 - half) * 128 + row;
        const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
        const int rows = p.gh * p.T;
        float* kfac = fact + h * 256;
        float* vfac = kfac + 128;
        int it = 0, pt = 0, piece = 0;
        while (pos < end && ok) {
            const int b = static_cast<int>(tile / p.rows_per_seq);
            const int rem = static_cast<int>(tile % p.rows_per_seq);
            const int hs = rem / p.mt;
            const int units = tree_units(p, tree_len(p, b));
            const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
            const int64_t out0 = (static_cast<int64_t>(b) * p.Hq + hs * p.gh) * p.T;  // first row of the group
            // the row tiles of a CTA share its rows evenly
            const int base = (rem % p.mt) * p.rpt, mine = min(p.rpt, rows - base);
            const int per = (mine + NM - 1) / NM;
            const int first = base + h * per, nrows = max(0, min(per, mine - h * per));
            const bool live = (warp % 4) * 32 < nrows;     // the two warps have a row
            const uint4* qg = reinterpret_cast<const uint4*>(p.Q + (out0 + first) * D);
            uint8_t* qt = q_s + h * C::QB;

            // Q as bf16: [D / 64][128 rows][128 B], 128-byte swizzle
            auto q_bf16 = [&]() {
                for (int e = half * 128 + row; e < 128 * (D / 8); e += 256) {
                    const int r = e / (D / 8), c = e % (D / 8);
                    const uint4 x = r < nrows ? __ldg(qg + e) : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(qt + (c / 8) * 16384 + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = x;
                }
            };
            float rf = 1.f;  // score factor of this thread's row
            // Q as e4m3 + e5m2 terms [128 rows][D B] each; D/8 lanes hold a row
            auto q_terms = [&]() {
                for (int e = half * 128 + row; e < 128 * (D / 8); e += 256) {
                    const int r = e / (D / 8), c = e % (D / 8);
                    const uint4 x = r < nrows ? __ldg(qg + e) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    float vv[8], top = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        vv[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
                        top = fmaxf(top, fabsf(vv[i]));
                    }
#pragma unroll
                    for (int o = 1; o < D / 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    // 2^(f - 127) brings the maximum to [224, 448): 448 = 1.75 * 2^8
                    const uint32_t tb = __float_as_uint(top);
                    const int f = min(253, 127 + 8 + 127 - static_cast<int>(tb >> 23) - ((tb & 0x7FFFFFu) > 0x600000u ? 1 : 0));
                    const float sc = __uint_as_float(static_cast<uint32_t>(f) << 23);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = vv[2 * i] * sc, bb = vv[2 * i + 1] * sc;
                        hi[i] = cvt_e4m3x2(a, bb);
                        const float2 hh = e4m3x2_f32(hi[i]);
                        lo[i] = cvt_e5m2x2(a - hh.x, bb - hh.y);
                        // an infinity saturates the first term: the second makes the score a NaN
                        if (isinf(a)) lo[i] = (lo[i] & 0xFF00u) | 0x7Fu;
                        if (isinf(bb)) lo[i] = (lo[i] & 0x00FFu) | 0x7F00u;
                    }
                    const int ch = c / 2;
                    const uint32_t off = D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) + 8 * (c & 1)
                                                  : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4) + 8 * (c & 1);
                    *reinterpret_cast<uint2*>(qt + off) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                    *reinterpret_cast<uint2*>(qt + 128 * D + off) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
                    if (c == 0) kfac[r] = __uint_as_float(static_cast<uint32_t>(254 - f) << 23);
                }
                named_bar_sync(group, 256);
                rf = kfac[row];
                named_bar_sync(group, 256);  // the table is the keys' from here on
            };
            auto q_ready = [&]() {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull);
            };
            if constexpr (E4M3)
                q_terms();
            else
                q_bf16();
            uint64_t bits = 0;  // the row's ancestors
            if (u1 == units && row < nrows)
                bits = __ldg(p.mask + static_cast<int64_t>(b) * p.T + (first + row) % p.T) &
                       (p.T == 64 ? ~0ull : (1ull << p.T) - 1ull);
            q_ready();

            float m = 0.f;      // the reference: a maximum so far, log2 units; 0 while there is none
            uint64_t l2 = 0ull; // the row's sum, in two halves
            bool fresh = true;
            int u = 0, uexp = 0;
            while (true) {
                // Warps that meet at barriers leave together when a wait ran out in one of them: e4m3, the row
                // tile's at a vote of their own; bf16, the row's two at the vote of the maxima, which is
                // taken a second time whenever the first is true, by a warp that does not know the slot too.
                if (ok) ok = mbar_wait(&sfull[bar_of(h, it)], par_of(it), p.status, kTreeDetail | 0x28u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if constexpr (E4M3) {
                    if (vote_any(group, 256, !ok)) {
                        ok = false;
                        break;
                    }
                } else if (!ok) {
                    if (live) {
                        vote_any(pair, 64, true);
                        vote_any(pair, 64, true);
                    }
                    break;
                }
                tc_fence_after();
                const int me = k.n % kTreeMeta;
                const int4 mt = meta[me];
                if (E4M3 && mt.x == kTileDraft) {
                    // this slot only says that the drafted tokens come: Q's buffer is free for the bf16 rows
                    q_bf16();
                    q_ready();
                    ++it;
                    ok = mbar_wait(&sfull[bar_of(h, it)], par_of(it), p.status, kTreeDetail | 0x29u);
                    if (vote_any(group, 256, !ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                if (mt.x == kTileEnd) {
                    if (!E4M3 && live && vote_any(pair, 64, false) && vote_any(pair, 64, false)) ok = false;
                    ++it;
                    k.next(p.nk);
                    break;
                }
                const bool draft = mt.x == kTileDraft;
                const bool whole_tile = !draft && mt.y == 64 && mt.z == 64;
                uint8_t* vt = vring + v.s * C::TILE;
                if (half == 0 && !whole_tile) {  // what follows writes V's tile: it has landed
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&vfull[v.s], v.par, p.status, kTreeDetail | 0x2Bu));
                }
                // V rows that do not count must not meet P's zeros as a NaN: each row tile clears them before its
                // own P (two row tiles: the same zeros twice)
                if (half == 0 && !draft && !whole_tile && (row & 63) >= (row < 64 ? mt.y : mt.z)) {
                    for (int c = 0; c < C::ROW / 16; ++c) {
                        uint8_t* z = vt + (E4M3 ? row * D + 16 * c : (c / 8) * 16384 + row * 128 + 16 * (c % 8));
                        *reinterpret_cast<uint4*>(z) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                if (half == 0 && draft && row < p.tp) {
                    // a drafted value that is not finite would reach every token through 0 * x: it is taken out
                    // here (by whichever row tile comes first) and given to the tokens that attend it at the end
                    uint32_t bad = 0;
                    for (int c = 0; c < D / 8; ++c) {
                        uint4* z = reinterpret_cast<uint4*>(vt + (c / 8) * 8192 + row * 128 + 16 * (c % 8));
                        uint32_t w[4] = {z->x, z->y, z->z, z->w};
                        uint32_t any = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u, any = 1;
                            if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0x0000FFFFu, any = 1;
                        }
                        if (row >= p.T) {
                            *z = make_uint4(0u, 0u, 0u, 0u);
                        } else if (any) {
                            *z = make_uint4(w[0], w[1], w[2], w[3]);
                            bad = 1;
                        }
                    }
                    if (bad) atomicOr(&dflag[piece & 1][row >> 5], 1u << (row & 31));
                }
                float kf = p.scale_log2;   // times the key's factor
                float uf = 1.f;            // what a new unit does to O
                if constexpr (E4M3) {
                    if (!draft) {
                        kf *= rf;
                        // the tile's factors, one key a thread; the unit is set by the largest V exponent
                        const bool counts = (row & 63) < (row < 64 ? mt.y : mt.z);
                        const uint32_t four = *reinterpret_cast<const uint32_t*>(exps + me * 256 + 128 + 4 * lane);
                        int top = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = 4 * lane + i;
                            if ((key & 63) < (key < 64 ? mt.y : mt.z)) top = max(top, static_cast<int>((four >> (8 * i)) & 0xFFu));
                        }
                        top = min(254, static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(top))));
                        if (fresh || top > uexp) {
                            uexp = top;
                            const int un = max(kTreeUMin, top - 127 + static_cast<int>(C::LAZY) - 15);
                            if (!fresh) uf = pow2i(max(-126, u - un));
                            u = un;
                        }
                        if (half == 0) {
                            const uint32_t ek = counts ? exps[me * 256 + row] : 0u;
                            kfac[row] = __uint_as_float(ek << 23);
                        } else {  // a row of exponent 255 stands for NaN (its bytes are zero)
                            const int ev = counts ? exps[me * 256 + 128 + row] : 0;
                            vfac[row] = __uint_as_float(ev == 255 ? 0x7FFFFFFFu : static_cast<uint32_t>(max(ev - u, 1)) << 23);
                        }
                        named_bar_sync(group, 256);
                    }
                }
                const uint32_t ts = tm + lanes + bar_of(h, it) * 128;
                const uint32_t to = tm + lanes + C::O_COL + h * 128;
                const int cb = 64 * half, ce = draft ? (half == 0 ? p.tp : 0) : cb + 64;  // this warp's columns
                const uint64_t kf2 = f2_pack(kf, kf);
                // 32 columns of S as scores (log2 units, -inf where masked)
                auto scores = [&](int c0, uint64_t (&x)[16]) {
                    uint32_t w[32];
                    tmem_ld32(ts + c0, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[i] = f2_mul(f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), kf2);
                    }
                    if (E4M3 && !draft) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = *reinterpret_cast<const float4*>(kfac + c0 + 4 * i);
                            x[2 * i] = f2_mul(x[2 * i], f2_pack(f.x, f.y));
                            x[2 * i + 1] = f2_mul(x[2 * i + 1], f2_pack(f.z, f.w));
                        }
                    }
                    if (!whole_tile) {
                        const int lim = draft ? 0 : (c0 < 64 ? mt.y : mt.z) - (c0 & 63);
                        const uint32_t on = draft ? static_cast<uint32_t>(bits >> (c0 & 63))
                                                  : lim >= 32 ? 0xFFFFFFFFu : lim <= 0 ? 0u : (1u << lim) - 1u;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float a, c;
                            f2_unpack(x[i], a, c);
                            x[i] = f2_pack((on >> (2 * i)) & 1u ? a : -INFINITY, (on >> (2 * i + 1)) & 1u ? c : -INFINITY);
                        }
                    }
                };
                if (live) {
                    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll 1
                    for (int c0 = cb; c0 < ce; c0 += 32) {
                        uint64_t x[16];
                        scores(c0, x);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float a, c, d, e;
                            f2_unpack(x[i], a, c);
                            f2_unpack(x[i + 1], d, e);
                            t0 = fmax3(t0, a, c);
                            t1 = fmax3(t1, d, e);
                        }
                    }
                    float top = fmaxf(t0, t1);
                    const bool over = fresh || top > m + C::LAZY || uf != 1.f;
                    if (vote_any(pair, 64, over)) {
                        if (!E4M3 && vote_any(pair, 64, false)) {
                            ok = false;
                            break;
                        }
                        *mine_x = top;
                        named_bar_sync(pair, 64);
                        top = fmaxf(top, *other_x);
                        // a row with nothing so far keeps 0 (its scores are all -inf and give 0)
                        const float now = fresh ? (top == -INFINITY ? 0.f : top) : fmaxf(m, top);
                        const float a = fresh || now == m ? 1.f : fast_exp2(m - now);
                        m = now;
                        if (!fresh) {
                            if constexpr (NM == 1) {
                                // (with two row tiles S itself waited for it)
                                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pvdone[bar_of(h, pt - 1)], par_of(pt - 1), p.status,
                                                                       kTreeDetail | 0x2Au));
                                tc_fence_after();
                            }
                            const float f = a * uf;
#pragma unroll 1
                            for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {  // half of O's columns each
                                uint32_t w[32];
                                tmem_ld32(to + c0, w);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
                                tmem_st32(to + c0, w);
                            }
                            tmem_wait_st();
                            l2 = f2_mul(l2, f2_pack(a, a));
                        }
                    }
                    const uint64_t nm2 = f2_pack(-m, -m);
                    const float pf = E4M3 && draft ? pow2i(min(127, max(-126, -u))) : 1.f;
                    const uint64_t pf2 = f2_pack(pf, pf);
#pragma unroll 1
                    for (int c0 = cb; c0 < ce; c0 += 32) {
                        uint64_t x[16];
                        scores(c0, x);
                        uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float a, c;
                            f2_unpack(f2_add(x[i], nm2), a, c);
                            x[i] = f2_pack(fast_exp2(a), fast_exp2(c));
                            if (i & 1)
                                s1 = f2_add(s1, x[i]);
                            else
                                s0 = f2_add(s0, x[i]);
                        }
                        l2 = f2_add(l2, f2_add(s0, s1));
                        if (E4M3 && !draft) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 f = *reinterpret_cast<const float4*>(vfac + c0 + 4 * i);
                                x[2 * i] = f2_mul(x[2 * i], f2_pack(f.x, f.y));
                                x[2 * i + 1] = f2_mul(x[2 * i + 1], f2_pack(f.z, f.w));
                            }
                            uint32_t t[3][8];
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                uint32_t hh[2], a1[2], a2[2], a3[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    float a, c;
                                    f2_unpack(x[2 * q + e], a, c);
                                    hh[e] = pack_f16x2(a, c);
                                    a1[e] = hh[e] & 0xFF00FF00u;
                                    hh[e] = sub_f16x2(hh[e], a1[e]);
                                    a2[e] = hh[e] & 0xFF00FF00u;
                                    a3[e] = sub_f16x2(hh[e], a2[e]) + 0x00800080u;  // rounded, not cut
                                }
                                t[0][q] = __byte_perm(a1[0], a1[1], 0x7531);
                                t[1][q] = __byte_perm(a2[0], a2[1], 0x7531);
                                t[2][q] = __byte_perm(a3[0], a3[1], 0x7531);
                            }
#pragma unroll
                            for (int i = 0; i < 3; ++i) tmem_st8(ts + c0 + 8 * i, t[i]);
                        } else {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float a, c;
                                if constexpr (E4M3) x[i] = f2_mul(x[i], pf2);
                                f2_unpack(x[i], a, c);
                                w[i] = pack_bf16x2(a, c);
                            }
                            tmem_st16(ts + c0, w);
                        }
                    }
                    tmem_wait_st();
                }
                fresh = false;
                tc_fence_before();
                fence_proxy_async_smem();
                if (E4M3 && !draft) named_bar_sync(group, 256);  // the table has been read
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[bar_of(h, pt)]);
                ++it;
                ++pt;
                k.next(p.nk);
                v.next(p.nv);
            }
            if (!ok) break;

            // ---- the piece's end (every product is complete): a thread writes its row
            const bool whole = unit == 0 && u1 == units;
            // partial slots: 2c for a piece that goes on with a row tile, 2c + 1 for one that begins it
            float* part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (unit == 0 ? 1 : 0)) * C::RM * (D + 2);
            const uint64_t odd = u1 == units ? dflag[piece & 1][0] | (static_cast<uint64_t>(dflag[piece & 1][1]) << 32) : 0ull;
            // rows of the CTA's row tile, in the order of the group
            const int at = h * per + row;
            if (live) {
                float la, lb;
                f2_unpack(l2, la, lb);
                *mine_x = la + lb;
                named_bar_sync(pair, 64);
                const float l = half == 0 ? *mine_x + *other_x : *other_x + *mine_x;  // the same order in both
                const float uo = E4M3 ? pow2i(min(127, max(-126, u))) : 1.f;
                const float f = whole ? (l == 0.f ? 0.f : uo / l) : uo;
                const bool mine_row = row < nrows;
                const int kvh = p.per_qhead ? hs / p.g : hs;
                const __nv_bfloat16* dv = p.DV + (static_cast<int64_t>(b) * p.Hkv + kvh) * p.T * D;
#pragma unroll 1
                for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
                    uint32_t w[32];
                    if (!fresh) {
                        tmem_ld32(tm + lanes + C::O_COL + h * 128 + c0, w);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = 0u;
                    }
                    float o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(w[i]) * f;
                    if (odd != 0) {
                        for (uint64_t left = odd & bits; left != 0; left &= left - 1) {
                            const int jd = __ffsll(static_cast<long long>(left)) - 1;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float y = __bfloat162float(dv[static_cast<int64_t>(jd) * D + c0 + i]);
                                if (!isfinite(y)) o[i] += y;
                            }
                        }
                    }
                    if (mine_row) {
                        if (whole) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                *reinterpret_cast<uint4*>(p.O + (out0 + base + at) * D + c0 + 8 * q) =
                                    make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                                               pack_bf16x2(o[8 * q + 4], o[8 * q + 5]), pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
                        } else {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<float4*>(part + at * D + c0 + 4 * q) =
                                    make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                        }
                    }
                }
                if (mine_row && half == 0) {
                    if (whole) {
                        if (p.lse != nullptr)
                            p.lse[out0 + base + at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                    } else {
                        part[C::RM * D + 2 * at] = l == 0.f ? -INFINITY : m;
                        part[C::RM * D + 2 * at + 1] = l;
                    }
                }
            }
            tc_fence_before();
            // the flags of the next piece: nobody reads the ones of the piece before any more (its successor's Q
            // was announced by every row tile)
            if (h == 0 && half == 0 && row < 2) dflag[(piece + 1) & 1][row] = 0;
            ++piece;
            pos += u1 - unit;
            unit = 0;
            ++tile;
        }
    }
    __syncthreads();
    if (warp == 8 * NM + 1) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

template <int D, bool E4M3, int NM>
static bool launch_many(TreeParams p, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dk,
                        const CUtensorMap& dv, cudaStream_t st, int32_t* launches) {
    using C = ManyCfg<D, E4M3, NM>;
    constexpr int budget = 225 * 1024;
    constexpr int fit = (budget - C::FIXED) / C::TILE;
    constexpr int slots = fit < 2 * kTreeMaxSlots ? fit : 2 * kTreeMaxSlots;
    static_assert(slots >= 4, "two slots of K and of V must fit");
    p.nk = slots / 2;
    p.nv = slots - p.nk;
    const int smem = C::FIXED + slots * C::TILE;
    static std::atomic<uint64_t> configured{0};
    if (!configure_smem_once(reinterpret_cast<const void*>(attn_tree_many_kernel<D, E4M3, NM>), smem, configured))
        return false;
    attn_tree_many_kernel<D, E4M3, NM><<<p.runs, C::THREADS, smem, st>>>(k, v, dk, dv, p);
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    return launch_tree_merge(p, D, C::RM, st, launches);
}

bool launch_attn_tree_many(TreeParams p, int D, bool e4m3, int rm, const void* K, const void* Kc, const void* Vc,
                           cudaStream_t st, int32_t* launches) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * p.cap, drows = static_cast<int64_t>(p.B) * p.Hkv * p.T;
    CUtensorMap k, v, dk, dv;
    if (!make_tmap_2d(&dk, K, drows, D, p.tp) || !make_tmap_2d(&dv, p.DV, drows, D, p.tp)) return false;
    if (e4m3 ? !make_tmap_2d_u8(&k, Kc, rows, D, 64) || !make_tmap_2d_u8(&v, Vc, rows, D, 64)
             : !make_tmap_2d(&k, Kc, rows, D, 64) || !make_tmap_2d(&v, Vc, rows, D, 64))
        return false;
#define PISA_MANY_CASE(DD, EE, NN) \
    if (D == DD && e4m3 == EE && rm == 128 * NN) return launch_many<DD, EE, NN>(p, k, v, dk, dv, st, launches);
    PISA_MANY_CASE(64, false, 1)
    PISA_MANY_CASE(64, false, 2)
    PISA_MANY_CASE(64, true, 1)
    PISA_MANY_CASE(64, true, 2)
    PISA_MANY_CASE(128, false, 1)
    PISA_MANY_CASE(128, false, 2)
    PISA_MANY_CASE(128, true, 1)
    PISA_MANY_CASE(128, true, 2)
#undef PISA_MANY_CASE
    return false;
}

}  // namespace pisa
