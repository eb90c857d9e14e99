// Tree attention for many rows: more than 16 drafted-token-and-head rows per selection row. The function and
// the cut into runs are in attn_tree.cu; here the tensor cores and the exponentials count as much as the
// bytes.
//
// Rows on the M side, 128 to a tile, one or two tiles in a CTA: S = Q K^T and O = P V with tcgen05, P read
// from TMEM, so a score costs no shared memory at all. (Keys on the M side, S^T = K Q^T and O^T = V^T P^T with
// 32 or 96 rows on N, was built first: K and V are then fetched as the 128-lane operand for every row tile,
// the values transposed at half the rate, and P goes through shared memory; 363 us for trees of 48 tokens of
// four heads over 8 ragged bf16 caches, 299 us in the first form of this one.) A row belongs to two softmax threads, one for each
// half of a tile's keys; the two warps meet in one vote a tile.
//
// A tile is 128 keys (two units of the cache, or the drafted tokens). Two passes over S in TMEM: the row's
// maximum (the kept one moves when one of the row's scores exceeds it by kManyLazy, and O with it, by the two warps), then
// the probabilities, written as operand A of P V over the columns of S that have been read. They are rounded to bf16,
// the type of the operand beside V, whose range a bf16 cache needs: O is 0.0023 from its 64-bit value where fp32
// probabilities leave 0.0017, the rounding of O itself (relative root mean squares, the trees below). Order of the
// MMA lane with two row tiles: S(0, g), P V(1, g - 1), S(1, g), P V(0, g): the softmax of one runs under the
// products of the other; with one row tile S has two buffers and the order is S(g), P V(g - 1).
//
// An e4m3 cache is turned into bf16 tiles on the way in: an e4m3 value times a power of two is a bf16 value
// (rounded once below bf16's smallest normal), and everything after is the same. For each ring one warp fetches
// the bytes, 32 rows a stage, and two or four converter warps write the swizzled tiles, some 65 instructions for
// 512 values. That is what bounds this form, together with the instruction cache: with the converters' loop
// unrolled four times and a copy of it for K and one for V, 32 tokens took 786 us and not 424 us (392 us since each
// warp takes whole steps). (With e4m3 operands in the products instead, P and Q need two and three 8-bit terms and
// every score a factor from a table: 469 us for 16 tokens.)
//
// Measured, with the join: trees of 48 tokens of 32 heads over 8 ragged bf16 caches up to 32,768 rows, 0.72 GB and
// 0.14 Tflop in 250 us (0.55 Pflop/s, 34 % of the measured peak). 64 caches of 8 heads, 64 blocks of 64 keys selected,
// tokens of four heads, bf16 (e4m3): 8 tokens 221 us, 16 tokens 227 us (326 us), 32 tokens 243 us (344 us), 64 tokens
// 396 us (555 us); the copy rate would be 167 us (86 us). What bounds it is the length of a row tile's own chain, S,
// softmax, P V, S again, of which the other row tile hides a part: tensor pipe 40 %, exponentials 31 %, issue 33 % of
// their peaks. In it the softmax makes two passes over S, each of blocking loads of 32 columns, with a vote of two warps
// between them. (The prefill kernel, with the same tiles and more keys a row, makes one pass against the kept maximum
// and reaches 0.96 Pflop/s; that form has not been tried here.) A quarter of the products of 48 tokens of four heads is
// empty rows, 192 in two tiles of 128. Steps of 64 keys with two buffers of S a row tile, which break the chain, cost
// more in the softmax than they hide (296 us for the trees).
// One elected lane issues the products: to the compiler a branch on the lane's number is not known to be one lane,
// and each product cost 90 cycles to issue (297 us).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pisa_device.cuh"
#include "pisa_tree.cuh"

namespace pisa {

constexpr int kManyStages = 8;     // e4m3: most stages of a ring
constexpr int kManySlots = 2;      // e4m3: slots of a ring
constexpr float kManyLazy = 8.f;    // log2 units a score may exceed the kept maximum by

template <int D, bool E4M3, int NM>
struct ManyCfg {
    static constexpr int TILE = 128 * 2 * D;             // one slot of a ring: K or V of a tile, bf16
    static constexpr int QB = 128 * 2 * D;               // one row tile of Q
    static constexpr int FIXED = 1024 + NM * (QB + 1024);  // 1024: [half][row] exchange
    static constexpr int RM = 128 * NM;
    // e4m3: converters of a ring, rows of a stage
    static constexpr int NC = NM == 2 ? 2 : 4, SR = 32, STAGE = SR * D + SR;
    static constexpr int THREADS = 256 * NM + 32 + (E4M3 ? 64 + 64 * NC : 32);
    static constexpr int O_COL = 256;                    // S: two of 128 columns (row tiles, or buffers)
};

// The producer warp (bf16): keeps the K and the V ring full by TMA. Every entry (a tile, or the end of a
// piece) takes a K slot and describes itself in meta[entry % kTreeMeta]; a tile takes a V slot too. K and V
// of a cache tile: [D / 64][128 rows][128 B]; of the drafted tokens: [D / 64][64 rows][128 B].
template <int D>
__device__ __forceinline__ void many_producer(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                              const CUtensorMap& tmDK, const CUtensorMap& tmDV, uint8_t* ring,
                                              uint8_t* vring, uint64_t* kfull, uint64_t* kempty, uint64_t* vfull,
                                              uint64_t* vempty, int4* meta, int64_t pos, int64_t end, int64_t tile,
                                              int unit) {
    constexpr int TILE = 128 * 2 * D;
    const int lane = threadIdx.x & 31;
    RingAt k, v;
    bool ok = true;
    if (lane == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmDK);
        prefetch_tmap(&tmDV);
    }
    auto issue = [&](int kind, int64_t plane, int len, int a0, int a1) {
        if (lane == 0) {
            ok = k.n < p.nk || mbar_wait(&kempty[k.s], k.par ^ 1u, p.status, kTreeDetail | 0x21u);
            if (ok) {
                uint8_t* kt = ring + k.s * TILE;
                uint64_t* kb = &kfull[k.s];
                const int halves = a1 >= 0 ? 2 : 1;
                const int dbytes = p.tp * 2 * D, dy = static_cast<int>(plane * p.T);
                meta[k.n % kTreeMeta] = make_int4(kind, min(64, len - a0), a1 >= 0 ? min(64, len - a1) : 0, 0);
                if (kind == kTileEnd) {
                    mbar_arrive(kb);
                } else if (kind == kTileDraft) {
                    mbar_arrive_expect_tx(kb, dbytes);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) tma_load_2d(kt + c * 8192, &tmDK, 64 * c, dy, kb);
                } else {
                    mbar_arrive_expect_tx(kb, halves * TILE / 2);
                    for (int h = 0; h < halves; ++h) {
                        const int y = static_cast<int>(plane * p.cap + (h == 0 ? a0 : a1));
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) tma_load_2d(kt + c * 16384 + h * 8192, &tmK, 64 * c, y, kb);
                    }
                }
                k.next(p.nk);
                if (kind != kTileEnd) {
                    ok = v.n < p.nv || mbar_wait(&vempty[v.s], v.par ^ 1u, p.status, kTreeDetail | 0x22u);
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
#pragma unroll
                                for (int c = 0; c < D / 64; ++c) tma_load_2d(vt + c * 16384 + h * 8192, &tmV, 64 * c, y, vb);
                            }
                        }
                        v.next(p.nv);
                    }
                }
            }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    };
    tree_entries<true>(p, pos, end, tile, unit, true, ok, issue);
    // every copy lands before the block ends, also when another role gave up (earlier uses of a slot were
    // complete before it was filled again)
    if (lane == 0) {
        for (int i = 0; i < p.nk && i < k.n; ++i) {
            k.s = k.s == 0 ? p.nk - 1 : k.s - 1;
            if (k.s == p.nk - 1) k.par ^= 1u;
            if (!mbar_wait(&kfull[k.s], k.par, p.status, kTreeDetail | 0x23u)) break;
        }
        for (int i = 0; i < p.nv && i < v.n; ++i) {
            v.s = v.s == 0 ? p.nv - 1 : v.s - 1;
            if (v.s == p.nv - 1) v.par ^= 1u;
            if (!mbar_wait(&vfull[v.s], v.par, p.status, kTreeDetail | 0x24u)) break;
        }
    }
}

// e4m3: for each ring, stages between the cache and the ring, SR rows with their exponents.
enum : int { kStepEnd = kTileEnd, kStepRows = kTileCache, kStepDraft = kTileDraft, kStepStop = 3 };
struct ManyStages {
    uint8_t* bytes;              // [p.ns][SR][D]
    uint8_t* exps;               // [p.ns][SR]
    uint64_t *full, *empty;
    int4* step;                  // kind | part of its tile << 4; keys of the two halves; use of the ring; plane
};

// The warp that fills the stages of the K ring or (is_v) of the V ring by bulk copy.
template <int D, int SR, int NC>
__device__ __forceinline__ void many_fetch(const TreeParams& p, const CUtensorMap* tmC, bool is_v, const ManyStages& g, int64_t pos, int64_t end,
                                           int64_t tile, int unit) {
    const int lane = threadIdx.x & 31;
    const uint8_t* exps = is_v ? p.v_exp : p.k_exp;
    RingAt r;
    int use = 0;  // of the ring, by the entry at hand
    bool ok = true;
    auto step = [&](int what, int keys, int plane, int64_t row, bool copy) {  // lane 0
        ok = ok && (r.n < p.ns || mbar_wait(&g.empty[r.s], r.par ^ 1u, p.status, kTreeDetail | (is_v ? 0x31u : 0x30u)));
        if (!ok) return;
        g.step[r.s] = make_int4(what, keys, use, plane);
        if (copy) {
            mbar_arrive_expect_tx(&g.full[r.s], SR * D + SR);
            tma_load_2d(g.bytes + r.s * SR * D, tmC, 0, static_cast<int>(row), &g.full[r.s]);
            bulk_load(g.exps + r.s * SR, exps + row, SR, &g.full[r.s]);
        } else {
            mbar_arrive(&g.full[r.s]);
        }
        r.next(p.ns);
    };
    auto issue = [&](int kind, int64_t plane, int len, int a0, int a1) {
        if (is_v && kind == kTileEnd) return;
        if (lane == 0) {
            const int n0 = min(64, len - a0), n1 = a1 >= 0 ? min(64, len - a1) : 0;
#pragma unroll 1
            for (int i = 0; i < 128 / SR; ++i) {
                const int r0 = i * SR;  // first row of the tile
                step(kind | i << 4, n0 | n1 << 16, static_cast<int>(plane), plane * p.cap + (r0 < 64 ? a0 + r0 : a1 + r0 - 64),
                     kind == kTileCache && (r0 < 64 ? r0 < n0 : r0 - 64 < n1));
            }
            ++use;
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    };
    tree_entries<true>(p, pos, end, tile, unit, !is_v, ok, issue);
    if (lane == 0) {
#pragma unroll 1
        for (int i = 0; i < NC; ++i) step(kStepStop, 0, 0, 0, false);
        // every copy lands before the block ends, also when another role gave up
        for (int i = 0; i < p.ns && i < r.n; ++i) {
            r.s = r.s == 0 ? p.ns - 1 : r.s - 1;
            if (r.s == p.ns - 1) r.par ^= 1u;
            if (!mbar_wait(&g.full[r.s], r.par, p.status, kTreeDetail | (is_v ? 0x33u : 0x32u))) break;
        }
    }
}

// Converter warp cw of the NC that turn the stages into the bf16 tiles of the K ring or (is_v) of the V ring:
// every NC-th step is its own (what a step costs beside its rows, 500 cycles, is then paid by one warp). Rows
// that do not count become zeros. The drafted tokens are bf16 and come by TMA. Every entry has 128 / SR steps,
// a multiple of NC, so that each warp takes part in every use of a slot and no parity of a barrier is passed
// over; the ring's full barriers count one arrival a step.
template <int D, int SR, int NC>
__device__ __forceinline__ void many_converter(const TreeParams& p, const CUtensorMap* tmD, bool is_v, int cw,
                                               const ManyStages& g, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                               int4* meta) {
    constexpr int TILE = 128 * 2 * D;
    constexpr int LPR = D / 16, RPI = 32 / LPR;          // lanes of a row, rows a warp takes at a time
    static_assert(128 / SR % NC == 0, "each warp sees every use");
    const int lane = threadIdx.x & 31, chunk = lane % LPR, rsub = lane / LPR;
    int drafts = -1;                                     // this warp's last use of the ring for drafted tokens
    bool ok = true;
    if (lane == 0) prefetch_tmap(tmD);
    RingAt r;
    for (int i = 0; i < cw; ++i) r.next(p.ns);
    while (true) {
        ok = mbar_wait(&g.full[r.s], r.par, p.status, kTreeDetail | (is_v ? 0x35u : 0x34u));
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const int4 what = g.step[r.s];
        const int kind = what.x & 15, part = what.x >> 4, use = what.z;
        if (kind == kStepStop) {
            // `use` is the number of uses: the slot's last one (its parity says whether all before are complete)
            if (drafts >= 0) drafts = use - 1 - (use - 1 - drafts) % kManySlots;
            break;
        }
        const int slot = use % kManySlots;
        ok = use < kManySlots ||
             mbar_wait(&empty[slot], (use / kManySlots & 1) ^ 1u, p.status, kTreeDetail | (is_v ? 0x22u : 0x21u));
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (lane == 0 && part == 0 && !is_v)
            meta[use % kTreeMeta] = make_int4(kind, what.y & 0xFFFF, what.y >> 16, 0);
        uint8_t* t = ring + slot * TILE;
        if (kind == kStepRows) {
            const int r0 = part * SR, n = r0 < 64 ? what.y & 0xFFFF : (what.y >> 16) + 64;  // rows below n count
            const uint8_t* src = g.bytes + r.s * SR * D;
            const uint8_t* ex = g.exps + r.s * SR;
#pragma unroll 1
            for (int row = rsub; row < SR; row += RPI) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                uint32_t e = 127;
                if (r0 + row < n) {
                    x = *reinterpret_cast<const uint4*>(src + row * D + ((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4));
                    e = ex[row];
                }
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[8], nan = 0;
                // seeeemmm as a bf16 with the exponent field eeee is the value times 2^-120, its subnormals too;
                // times 2^(e - 7) then
                const uint32_t f = (e + 120u) << 7, f1 = f | (f << 16);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t y = __byte_perm(w[c / 2], 0u, (c & 1) ? 0x3424 : 0x1404);
                    o[c] = bf16x2_mul((y & 0x80008000u) | ((y >> 4) & 0x07F007F0u), f1);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) nan |= (w[c] & 0x7F7F7F7Fu) + 0x01010101u;
                // 2^(e - 7) is no bf16 above e = 134; a byte that is a NaN is none of the above
                if (e > 134u || (nan & 0x80808080u) != 0u) {
                    const float g = __uint_as_float(e << 23);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t v = c == 0 ? x.x : c == 1 ? x.y : c == 2 ? x.z : x.w;
                        const float2 lo = e4m3x2_f32(v & 0xFFFFu), hi = e4m3x2_f32(v >> 16);
                        const uint32_t y0 = pack_bf16x2(lo.x * g, lo.y * g), y1 = pack_bf16x2(hi.x * g, hi.y * g);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            o[2 * q] = q == c ? y0 : o[2 * q];
                            o[2 * q + 1] = q == c ? y1 : o[2 * q + 1];
                        }
                    }
                }
                uint8_t* dst = t + (chunk / 4) * 16384 + (r0 + row) * 128;
                const int c = 2 * (chunk % 4);
                *reinterpret_cast<uint4*>(dst + ((c ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(dst + (((c + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&g.empty[r.s]);
            if (kind == kStepDraft && part == 0) {
                drafts = use;
                mbar_arrive_expect_tx(&full[slot], p.tp * 2 * D);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) tma_load_2d(t + c * 8192, tmD, 64 * c, what.w * p.T, &full[slot]);
            } else {
                mbar_arrive(&full[slot]);
            }
        }
        for (int i = 0; i < NC; ++i) r.next(p.ns);
    }
    // the drafted tokens' copies land before the block ends, also when another role gave up
    if (lane == 0 && drafts >= 0)
        mbar_wait(&full[drafts % kManySlots], drafts / kManySlots & 1, p.status, kTreeDetail | (is_v ? 0x24u : 0x23u));
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
    uint8_t* q_s = vring + p.nv * C::TILE;               // [row tile][D / 64][128 rows][128 B]
    float* xch = reinterpret_cast<float*>(q_s + NM * C::QB);  // [row tile][half][128]
    uint8_t* stages = reinterpret_cast<uint8_t*>(xch) + NM * 1024;  // e4m3: of K, of V
    __shared__ __align__(8) uint64_t kfull[kTreeMaxSlots], kempty[kTreeMaxSlots], vfull[kTreeMaxSlots],
        vempty[kTreeMaxSlots], rfull[2][kManyStages], rempty[2][kManyStages], sfull[2], pfull[2], pvdone[2], qfull, done;
    __shared__ int4 step[2][kManyStages];
    __shared__ int4 meta[kTreeMeta];  // kind, keys that count in the two halves
    __shared__ uint32_t tmem_slot, dflag[2][2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join finds its place as CTAs end
    const TreeJob job = tree_job(p);
    if (static_cast<int64_t>(blockIdx.x) >= job.runs) return;
    int64_t pos = job.begin(blockIdx.x);
    const int64_t end = job.begin(blockIdx.x + 1);
    int64_t tile;
    int unit;
    tree_find(p, pos, tile, unit);
    if (tid == 0) {
        for (int i = 0; i < p.nk; ++i) {
            mbar_init(&kfull[i], E4M3 ? 128 / C::SR : 1);
            mbar_init(&kempty[i], 1);
        }
        for (int i = 0; i < p.nv; ++i) {
            mbar_init(&vfull[i], E4M3 ? 128 / C::SR : 1);
            mbar_init(&vempty[i], 1);
        }
        for (int i = 0; i < p.ns; ++i)
            for (int x = 0; x < 2; ++x) {
                mbar_init(&rfull[x][i], 1);
                mbar_init(&rempty[x][i], 1);
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
    if (warp == 8 * NM) tmem_alloc(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    bool ok = true;       // cleared by a wait that ran out: nothing more is waited for
    RingAt k, v;          // K ring (tiles and piece ends), V ring (tiles)
    // Row tile h and number n of a tile (or of an S slot) -> barrier, its parity, and the columns of S.
    auto bar_of = [](int h, int n) { return NM == 2 ? h : n & 1; };
    auto par_of = [](int n) { return static_cast<uint32_t>((NM == 2 ? n : n >> 1) & 1); };

    if (warp > 8 * NM) {
        // ------------------------------------------------ tiles
        if constexpr (E4M3)
        {
            // one copy of the code for K and V: the roles' code together is more than the instruction cache holds
            const int w = warp - 8 * NM - 1;
            const bool is_v = w < 2 ? w == 1 : w - 2 >= C::NC;
            const int x = is_v ? 1 : 0;
            const int n = p.ns * C::SR;  // rows of a ring's stages; the bytes of both rings (each stage at a multiple
                                         // of 1024, the swizzle's period), then the exponents
            const ManyStages g = {stages + x * n * D, stages + 2 * n * D + x * n, rfull[x], rempty[x], step[x]};
            if (w < 2)
                many_fetch<D, C::SR, C::NC>(p, is_v ? &tmV : &tmK, is_v, g, pos, end, tile, unit);
            else
                many_converter<D, C::SR, C::NC>(p, is_v ? &tmDV : &tmDK, is_v, w - 2 - x * C::NC, g, is_v ? vring : ring,
                                                is_v ? vfull : kfull, is_v ? vempty : kempty, meta);
        } else {
            many_producer<D>(p, tmK, tmV, tmDK, tmDV, ring, vring, kfull, kempty, vfull, vempty, meta, pos, end, tile, unit);
        }
    } else if (warp == 8 * NM) {
        // ------------------------------------------------ MMA
        if (elect_one()) {
            const uint32_t q0 = smem_u32(q_s);
            int it = 0, tn = 0;       // S slots so far, and tiles among them
            int pn = 0, pit = 0;      // tiles whose P V was issued for every row tile; the S slot of the next one
            bool pend = false;        // P V of the tile before is still to be issued (two row tiles: for tile 1)
            bool pdraft = false;      // and that tile is the drafted tokens;
            int psteps = 0;           // its steps
            uint32_t fresh = 3u;      // bit h: the next P V of row tile h begins O
            uint32_t qpar = 0;
            bool issued = false;
            // S of row tile h from the K slot at hand. (Loops stay loops here: the roles' code together is more
            // than the instruction cache holds, and what waits in this lane is seldom its own issue.)
            auto qk = [&](int h, bool draft) {
                const uint32_t kt = smem_u32(ring + k.s * C::TILE), qt = q0 + h * C::QB;
                const uint32_t d = tm + bar_of(h, it) * 128;
                const uint32_t sub = draft ? 8192 : 16384;
                const uint64_t a = smem_desc_sw128(qt, 16, 1024), b = smem_desc_sw128(kt, 16, 1024);
                const uint32_t id = idesc_bf16_f32(128, draft ? p.tp : 128, 0, 0);
#pragma unroll
                for (int n = 0; n < D / 16; ++n)
                    mma_bf16_ss(d, desc_at(a, (n / 4) * 16384 + (n % 4) * 32), desc_at(b, (n / 4) * sub + (n % 4) * 32), id,
                                n > 0 ? 1u : 0u);
                mma_commit(&sfull[bar_of(h, it)]);
            };
            // P V of row tile h for tile number n (S slot sit) from the V slot at hand, 16 keys a step
            auto pv = [&](int h, int n, int sit, bool draft, int steps) {
                ok = mbar_wait(&pfull[bar_of(h, n)], par_of(n), p.status, kTreeDetail | 0x25u) &&
                     mbar_wait(&vfull[v.s], v.par, p.status, kTreeDetail | 0x26u);
                if (!ok) return;
                tc_fence_after();
                const uint32_t vt = smem_u32(vring + v.s * C::TILE);
                const uint32_t a = tm + bar_of(h, sit) * 128, d = tm + C::O_COL + h * 128;
                const uint64_t b = smem_desc_sw128(vt, draft ? 8192 : 16384, 1024);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < steps) mma_bf16_ts(d, a + 32 * (i / 2) + 8 * (i % 2), desc_at(b, i * 2048), idesc_bf16_f32(128, D, 0, 1),
                                i > 0 ? 1u : !(fresh >> h & 1u));
                fresh &= ~(1u << h);
                mma_commit(&pvdone[bar_of(h, n)]);
            };
            while (pos < end && ok) {
                const int b = static_cast<int>(tile / p.rows_per_seq);
                const int units = tree_units(p, tree_len(p, b));
                const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
                ok = mbar_wait(&qfull, qpar, p.status, kTreeDetail | 0x29u);
                qpar ^= 1u;
                fresh = 3u;
                bool over = false;
                while (ok && !over) {
                    ok = mbar_wait(&kfull[k.s], k.par, p.status, kTreeDetail | 0x2Cu);
                    if (!ok) break;
                    const int4 mt = meta[k.n % kTreeMeta];
                    const bool draft = mt.x == kTileDraft;
                    const int steps = draft ? p.tp / 16 : mt.z > 0 ? 4 + (mt.z + 15) / 16 : (mt.y + 15) / 16;
                    over = mt.x == kTileEnd;
                    issued = true;
                    // one step for each row tile: its S, then the P V that is due (two row tiles: of the other one)
#pragma unroll 1
                    for (int h = 0; h < (over ? 1 : NM) && ok; ++h) {
                        if (!over) {
                            // S goes where an earlier tile's P is read from: two row tiles, the tile before's; one
                            // row tile, that of two before
                            const int back = NM == 2 ? 1 : 2;
                            if (tn >= back)
                                ok = mbar_wait(&pvdone[bar_of(h, tn - back)], par_of(tn - back), p.status, kTreeDetail | 0x2Du);
                            if (!ok) break;
                            tc_fence_after();
                            qk(h, draft);
                            if (h == NM - 1) mma_commit(&kempty[k.s]);
                        }
                        const bool due = h == 0;  // of the tile before, the last product of its V slot
                        if (due && !pend) continue;
                        pv(due ? NM - 1 : 0, due ? pn : tn, due ? pit : it, due ? pdraft : draft, due ? psteps : steps);
                        if (ok && due) {
                            mma_commit(&vempty[v.s]);
                            v.next(p.nv);
                            ++pn;
                            pend = false;
                        }
                    }
                    if (!ok) break;
                    if (over) {  // an S slot without scores, after every product so far: the softmax may read O
                        mma_commit(&sfull[bar_of(0, it)]);
                        if (NM == 2) mma_commit(&sfull[1]);
                        mbar_arrive(&kempty[k.s]);
                    } else {
                        pend = true;
                        pdraft = draft;
                        psteps = steps;
                        pit = it;
                        ++tn;
                    }
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
        const uint32_t pair = 1 + 4 * h + warp % 4;  // barrier of the row's two warps
        float* mine_x = xch + h * 256 + half * 128 + row;
        const float* other_x = xch + h * 256 + (1 - half) * 128 + row;
        const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
        const int rows = p.gh * p.T;
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

            // Q: [D / 64][128 rows][128 B], 128-byte swizzle
            for (int e = half * 128 + row; e < 128 * (D / 8); e += 256) {
                const int r = e / (D / 8), c = e % (D / 8);
                const uint4 x = r < nrows ? __ldg(qg + e) : make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(qt + (c / 8) * 16384 + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = x;
            }
            uint64_t bits = 0;  // the row's ancestors
            if (u1 == units && row < nrows)
                bits = __ldg(p.mask + static_cast<int64_t>(b) * p.T + (first + row) % p.T) &
                       (p.T == 64 ? ~0ull : (1ull << p.T) - 1ull);
            // the MMA lane saw the piece before to its end (the slot that ends a piece comes through it)
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&qfull);

            float m = kTreeNone;  // the reference: a maximum so far, log2 units
            uint64_t l2 = 0ull; // the row's sum, in two halves
            bool fresh = true;
            while (true) {
                // The row's two warps leave together when a wait ran out in one of them: the vote of the maxima
                // is taken a second time whenever the first is true, by a warp that does not know the slot too.
                if (ok) ok = mbar_wait(&sfull[bar_of(h, it)], par_of(it), p.status, kTreeDetail | 0x28u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) {
                    if (live) {
                        vote_any(pair, 64, true);
                        vote_any(pair, 64, true);
                    }
                    break;
                }
                tc_fence_after();
                const int4 mt = meta[k.n % kTreeMeta];
                if (mt.x == kTileEnd) {
                    if (live && vote_any(pair, 64, false) && vote_any(pair, 64, false)) ok = false;
                    ++it;
                    k.next(p.nk);
                    break;
                }
                const bool draft = mt.x == kTileDraft;
                const bool whole_tile = !draft && mt.y == 64 && mt.z == 64;
                uint8_t* vt = vring + v.s * C::TILE;
                if (draft || (!E4M3 && !whole_tile)) {  // what follows writes V's tile: it has landed
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&vfull[v.s], v.par, p.status, kTreeDetail | 0x2Bu));
                    // (two row tiles do the same twice: either may come first)
                    const int t = half * 128 + row;
                    if (draft) {
                        // a drafted value that is not finite would reach every token through 0 * x: it is taken out
                        // here and given to the tokens that attend it at the end; rows past the tokens become zeros
#pragma unroll 1
                        for (int e = t; e < p.tp * (D / 8); e += 256) {
                            const int r = e / (D / 8), c = e % (D / 8);
                            uint4* z = reinterpret_cast<uint4*>(vt + (c / 8) * 8192 + r * 128 + 16 * (c % 8));
                            uint32_t w[4] = {z->x, z->y, z->z, z->w};
                            uint32_t any = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u, any = 1;
                                if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0x0000FFFFu, any = 1;
                            }
                            if (r >= p.T) {
                                *z = make_uint4(0u, 0u, 0u, 0u);
                            } else if (any) {
                                *z = make_uint4(w[0], w[1], w[2], w[3]);
                                atomicOr(&dflag[piece & 1][r >> 5], 1u << (r & 31));
                            }
                        }
                    } else {
                        // V rows that do not count, in the steps that are taken, must not meet P's zeros as a NaN
                        const int e0 = mt.z > 0 ? 64 : (mt.y + 15) & ~15, e1 = (mt.z + 15) & ~15;
#pragma unroll 1
                        for (int e = t; e < (e0 - mt.y + e1 - mt.z) * (D / 8); e += 256) {
                            const int i = e / (D / 8), c = e % (D / 8);
                            const int r = i < e0 - mt.y ? mt.y + i : 64 + mt.z + i - (e0 - mt.y);
                            *reinterpret_cast<uint4*>(vt + (c / 8) * 16384 + r * 128 + 16 * (c % 8)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                const uint32_t ts = tm + lanes + bar_of(h, it) * 128;
                const uint32_t to = tm + lanes + C::O_COL + h * 128;
                const int cb = 64 * half, ce = draft ? (half == 0 ? p.tp : 0) : cb + 64;  // this warp's columns
                const uint64_t kf2 = f2_pack(p.scale_log2, p.scale_log2);
                // 32 columns of S as scores (log2 units, -inf where masked)
                auto scores = [&](int c0, uint64_t (&x)[16]) {
                    uint32_t w[32];
                    tmem_ld32(ts + c0, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[i] = f2_mul(f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), kf2);
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
                    if (vote_any(pair, 64, fresh || top > m + kManyLazy)) {
                        if (vote_any(pair, 64, false)) {
                            ok = false;
                            break;
                        }
                        *mine_x = top;
                        named_bar_sync(pair, 64);
                        top = fmaxf(top, *other_x);
                        // only a row that exceeds its own reference moves it: what another row attends changes no bit of
                        // this one
                        const float now = fresh ? fmaxf(m, top) : top > m + kManyLazy ? top : m;
                        const float a = fresh || now == m ? 1.f : fast_exp2(m - now);
                        m = now;
                        if (!fresh) {
                            if constexpr (NM == 1) {
                                // (with two row tiles S itself waited for it)
                                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pvdone[bar_of(h, pt - 1)], par_of(pt - 1), p.status,
                                                                       kTreeDetail | 0x2Au));
                                tc_fence_after();
                            }
#pragma unroll 1
                            for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {  // half of O's columns each
                                uint32_t w[32];
                                tmem_ld32(to + c0, w);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * a);
                                tmem_st32(to + c0, w);
                            }
                            tmem_wait_st();
                            l2 = f2_mul(l2, f2_pack(a, a));
                        }
                    }
                    const uint64_t nm2 = f2_pack(-m, -m);
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
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float a, c;
                            f2_unpack(x[i], a, c);
                            w[i] = pack_bf16x2(a, c);
                        }
                        tmem_st16(ts + c0, w);
                    }
                    tmem_wait_st();
                }
                fresh = false;
                tc_fence_before();
                fence_proxy_async_smem();
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
                const float f = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
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
    if (warp == 8 * NM) {
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
    constexpr int most = E4M3 ? 2 * kManySlots : 2 * kTreeMaxSlots, slots = fit < most ? fit : most;
    static_assert(slots >= 4, "two slots of K and of V must fit");
    constexpr int spare = (budget - C::FIXED - slots * C::TILE) / (2 * C::STAGE);
    constexpr int ns = !E4M3 ? 0 : spare < kManyStages ? spare : kManyStages;
    static_assert(!E4M3 || ns >= 2, "two stages of each must fit");
    p.nk = slots / 2;
    p.nv = slots - p.nk;
    p.ns = ns;
    constexpr int smem = C::FIXED + slots * C::TILE + 2 * ns * C::STAGE;
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
    if (e4m3 ? !make_tmap_2d_u8(&k, Kc, rows, D, 32) || !make_tmap_2d_u8(&v, Vc, rows, D, 32)
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
