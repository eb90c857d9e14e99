// Tree attention for few rows: at most 16 drafted-token-and-head rows per selection row (one token of a
// group of four or eight heads is 4 or 8), or two tiles of such (e4m3, up to 32 rows). The function, the cut into runs and the treatment of the
// drafted tokens are those of attn_tree.cu; here nothing but the bytes of the cache should count.
//
// Bound: the bytes of the cache, each read once. One warp takes 16 keys of every unit of 64 on its own,
// with mma.sync m16n8k16: no barrier between warps, four copies of the softmax state per CTA that
// meet when a piece ends. (On tcgen05 the same step is a chain of hand-overs per tile, S, softmax, P, O,
// which few rows cannot fill: 160 to 185 us against 144 us for a first form of this kernel with the
// rows on the M side, for one token over 64 caches of 128K rows, 64 selected 8-bit blocks.)
//
// Keys and dims on the M side. S^T = K Q^T (16 keys x 16 dims x 8 rows a product) and O^T = V^T P^T
// (16 dims x 16 keys x 8 rows): rows are the N side, 8 to a tile, so a group of four heads wastes half a
// tile and not three quarters, and a softmax thread has two rows and two keys. P^T goes from the
// accumulators of S^T to an operand of O^T by two 8 x 8 register transposes.
//
// e4m3 rows become fp16 in registers, two values an instruction:
//   * Q is scaled by a power of two per row to a maximum in [2^14, 2^15) and rounded to fp16, which
//     keeps bf16's 8 bits for values down to 2^-29 of the row's largest.
//   * K's row exponent and Q's come back as an exact factor of the score, in fp32.
//   * V's row exponent goes into P. A key's weight is p 2^(e - 127), and every row has a power of two f of its own, set by
//     the largest weight that it has met: P' = p f 2^(e - 127), 2^3 to 2^4 for that key and at most 2^15 for any, O in
//     units of 1 / f. In fp16 P' keeps 11 bits down to 2^-17 of the largest weight and is a multiple of 2^-27 of it
//     below: off by 2^-28 of the largest entry that another row adds, where that row's own rounding in the cache is
//     up to 2^-19 of it (half of e4m3's smallest step against 448). (With one unit a warp, set by the largest exponent
//     whatever its probability, a value row of 2^34 times the others hid them all, at any weight. With a second
//     exponential a score, of its weight, four tokens below take 160 us, and eight 296 us and not 276 us.)
//   * ldmatrix hands out byte pairs: in Q K^T the dims of a 16-dim chunk take the order that the bytes
//     come in (any order does), in V^T P^T the even dims of a chunk are rows 0-7 of the product and the
//     odd ones rows 8-15.
// A bf16 cache takes P as bf16 (range of V); so do the drafted tokens, whose largest magnitude stands for the exponent.
//
// Measured (64 caches of 8 heads of 128, 64 selected blocks of 64 keys and 63 keys of tail, four query heads each):
// one token over e4m3 0.55 GB in 99 us with the join, 5.5 TB/s (84 % of the copy rate). Four tokens (16 rows)
// 148 us, bound by issue. Over bf16 1.09 GB: one token 179 us, 6.1 TB/s (93 %), four tokens 184 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pisa_device.cuh"
#include "pisa_tree.cuh"

namespace pisa {

constexpr float kFewLazy = 8.0f;    // log2 units a score may exceed the kept maximum by
constexpr float kFewTop = 15.0f;    // log2 of the largest P': fp16 ends below 2^16
constexpr float kFewUnit = 4.0f;    // log2 of P' of the largest weight when f is set, rounded down: weights may rise by 2^11,
                                    // exponents by 3 above that key's, before it is looked at again
constexpr float kFewMaxF = 100.0f;  // largest log2 f: P' of a drafted token is a finite bf16
constexpr float kFewDraftMin = -90.0f;  // smallest exponent of a drafted row
constexpr int kFewStages = 8;       // most stages of the ring
constexpr int kFewThreads = 160;    // four consumer warps and the producer

__device__ __forceinline__ void few_ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void few_ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t few_transpose(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
template <bool F16>
__device__ __forceinline__ void few_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// byte offset of 16-byte chunk `c` of row `row` in a tile of 128-byte (64-byte) swizzled rows
__device__ __forceinline__ uint32_t few_at128(int row, int c) {
    return static_cast<uint32_t>(row * 128 + ((c ^ (row & 7)) << 4));
}
template <int D>
__device__ __forceinline__ uint32_t few_at_e4m3(int row, int c) {
    return D == 128 ? few_at128(row, c) : static_cast<uint32_t>(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}

template <int D, bool E4M3, int NT>
struct FewCfg {
    static constexpr int ROW = E4M3 ? D : 2 * D;
    static constexpr int TILE = 64 * ROW;                // K (or V) of one unit
    static constexpr int STAGE = 2 * TILE;
    static constexpr int EXPS = E4M3 ? 128 : 0;          // exponent bytes of K and of V
    static constexpr int DRAFT = 16 * 2 * D;             // drafted K (or V), 16 rows
    static constexpr int RM = 8 * NT;
    static constexpr int CH = 32 / NT;                   // dims that meet at a time when a piece ends
    static constexpr int FIXED = 1024 + 2 * DRAFT + 4 * RM * (CH + 2) * 4;
    // three CTAs on an SM where two stages a CTA or more remain (the decode step above: 101 us, 112 with two
    // CTAs of five stages), else two
    static constexpr int CTAS = E4M3 && NT == 1 ? 3 : 2;
};

// One warp's state: for its rows 2 (lane % 4), + 1 of every row tile of 8 the reference that its
// probabilities are taken against (a maximum so far, log2 units; kTreeNone while there is none; whole for e4m3, so that
// rescaling is exact) and the sum over its keys; O^T: tile j is dims 16 j + lane / 4 (+ 8) (e4m3: 16 j + 2 (lane / 4),
// + 1); e4m3: f, and the largest exponent byte with which no P' of a score below ref + kFewLazy passes its largest.
template <int D, bool E4M3, int NT>
struct FewState {
    float o[NT][D / 16][4];
    float ref[NT][2], l[NT][2];
    float f[E4M3 ? NT : 1][2];
    int emax;
    bool fresh;   // no key yet
};

__device__ __forceinline__ float few_rows_max(float x) {  // over the keys of a row
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
}
__device__ __forceinline__ float few_log2(float f) {  // of a power of two
    return static_cast<float>(static_cast<int>(__float_as_uint(f) >> 23) - 127);
}

// Scores of 16 keys (log2 units, -inf where masked; [0], [1]: this thread's first key, [2], [3]: its
// second) -> what multiplies the keys' values: probabilities, or (e4m3) P', with e0 and e1 the exponent bytes of the
// two keys' values (255: the row stands for NaN). Drafted tokens (DRAFT): w0 and w1 are their exponents, which their
// values hold themselves. A row's reference or f moves, and its sum or O with it, when one of its own scores or weights
// asks for it: what another row attends changes no bit of this one.
template <int D, bool E4M3, int NT, bool DRAFT>
__device__ __forceinline__ void few_softmax(FewState<D, E4M3, NT>& s, float (&x)[NT][4], int e0, int e1, float w0, float w1) {
    bool over = s.fresh || (E4M3 && (DRAFT || max(e0, e1) > s.emax));
#pragma unroll
    for (int t = 0; t < NT; ++t)
        over = over || fmaxf(x[t][0], x[t][2]) > s.ref[t][0] + kFewLazy || fmaxf(x[t][1], x[t][3]) > s.ref[t][1] + kFewLazy;
    if (__any_sync(0xFFFFFFFFu, over)) {
        if constexpr (E4M3 && !DRAFT) {
            w0 = e0 == 255 ? __uint_as_float(0x7FC00000u) : static_cast<float>(e0 - 127);
            w1 = e1 == 255 ? __uint_as_float(0x7FC00000u) : static_cast<float>(e1 - 127);
        }
        float least = INFINITY;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float top = few_rows_max(fmaxf(x[t][e], x[t][2 + e]));
                const float old = s.ref[t][e];
                float now;
                if constexpr (E4M3) {
                    const float wtop = few_rows_max(fmaxf(x[t][e] + w0, x[t][2 + e] + w1));
                    const float lf = few_log2(s.f[t][e]);
                    const bool none = old == kTreeNone;
                    const bool move = none || top > old + kFewLazy || wtop - old + lf > kFewTop;
                    now = move ? fmaxf(old, ceilf(top)) : old;
                    // the unit of O stays, unless a weight is larger than the one that set it
                    const float stay = none ? kFewMaxF : fminf(kFewMaxF, lf + (now - old));
                    const float lfn = move ? fmaxf(-126.f, fminf(stay, floorf(kFewUnit - (wtop - now)))) : lf;
                    a[e] = none ? 1.f : fast_exp2((old - now) + (lfn - lf));
                    s.l[t][e] *= none ? 1.f : fast_exp2(old - now);
                    s.f[t][e] = __uint_as_float(static_cast<uint32_t>(static_cast<int>(lfn) + 127) << 23);
                    least = fminf(least, kFewTop - kFewLazy - lfn);
                } else {
                    now = s.fresh ? fmaxf(kTreeNone, top) : top > old + kFewLazy ? top : old;
                    a[e] = s.fresh || now == old ? 1.f : fast_exp2(old - now);
                    s.l[t][e] *= a[e];
                }
                s.ref[t][e] = now;
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                s.o[t][j][0] *= a[0];
                s.o[t][j][1] *= a[1];
                s.o[t][j][2] *= a[0];
                s.o[t][j][3] *= a[1];
            }
        }
        s.fresh = false;
        if constexpr (E4M3) {
            least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, 1));
            least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, 2));
            s.emax = 127 + static_cast<int>(least);
        }
    }
    const float g0 = __uint_as_float(static_cast<uint32_t>(e0) << 23), g1 = __uint_as_float(static_cast<uint32_t>(e1) << 23);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            x[t][e] = fast_exp2(x[t][e] - s.ref[t][e]);
            x[t][2 + e] = fast_exp2(x[t][2 + e] - s.ref[t][e]);
            s.l[t][e] += x[t][e] + x[t][2 + e];
            if constexpr (E4M3) {  // (p f first: f 2^(e - 127) may be no fp32)
                x[t][e] *= s.f[t][e];
                x[t][2 + e] *= s.f[t][e];
                if constexpr (!DRAFT) {
                    x[t][e] *= g0;
                    x[t][2 + e] *= g1;
                }
            }
        }
    }
}

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kFewThreads, (FewCfg<D, E4M3, NT>::CTAS))
    attn_tree_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                         const TreeParams p) {
    using C = FewCfg<D, E4M3, NT>;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* dk_s = ring + p.nk * C::STAGE;              // drafted K, then V: [D / 64][16][128 B]
    float* comb = reinterpret_cast<float*>(dk_s + 2 * C::DRAFT);       // [warp][row][CH]
    float* cml = comb + 4 * C::RM * C::CH;                             // [warp][row][m, l]
    uint8_t* exps = reinterpret_cast<uint8_t*>(cml + 4 * C::RM * 2);   // [stage][K 64, V 64]
    __shared__ __align__(8) uint64_t full[kFewStages], empty[kFewStages], dfull, dempty;
    __shared__ int meta[kFewStages];   // keys of the stage's tile that count; 0: the piece ends

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
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 4);
        }
        mbar_init(&dfull, 1);
        mbar_init(&dempty, 4);
        fence_barrier_init();
    }
    __syncthreads();

    int s = 0;            // ring stage, and the parity of its current use
    uint32_t par = 0, dpar = 0;
    bool ok = true;       // cleared by a wait that ran out: nothing more is waited for
    auto advance = [&]() {
        if (++s == p.nk) {
            s = 0;
            par ^= 1u;
        }
    };

    if (warp == 4) {
        // ------------------------------------------------ producer
        int used = 0, drafts = 0;
        if (lane == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            prefetch_tmap(&tmDK);
            prefetch_tmap(&tmDV);
        }
        auto issue = [&](int kind, int64_t plane, int len, int a, int) {
            if (kind == kTileDraft) {  // the drafted tokens, in a buffer of their own
                if (elect_one()) {
                    ok = drafts == 0 || mbar_wait(&dempty, dpar ^ 1u, p.status, kTreeDetail | 0x12u);
                    if (ok) {
                        mbar_arrive_expect_tx(&dfull, 2 * C::DRAFT);
                        const int y = static_cast<int>(plane * p.T);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            tma_load_2d(dk_s + c * 2048, &tmDK, 64 * c, y, &dfull);
                            tma_load_2d(dk_s + C::DRAFT + c * 2048, &tmDV, 64 * c, y, &dfull);
                        }
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (ok) {
                    ++drafts;
                    dpar ^= 1u;
                }
                return;
            }
            if (elect_one()) {
                ok = used < p.nk || mbar_wait(&empty[s], par ^ 1u, p.status, kTreeDetail | 0x11u);
                if (ok && kind == kTileEnd) {  // a slot without a tile
                    meta[s] = 0;
                    mbar_arrive(&full[s]);
                } else if (ok) {
                    meta[s] = min(64, len - a);
                    uint8_t* kt = ring + s * C::STAGE;
                    const int64_t krow = plane * p.cap + a;
                    const int y = static_cast<int>(krow);
                    mbar_arrive_expect_tx(&full[s], C::STAGE + C::EXPS);
                    if constexpr (E4M3) {
                        tma_load_2d(kt, &tmK, 0, y, &full[s]);
                        tma_load_2d(kt + C::TILE, &tmV, 0, y, &full[s]);
                        bulk_load(exps + s * 128, p.k_exp + krow, 64, &full[s]);
                        bulk_load(exps + s * 128 + 64, p.v_exp + krow, 64, &full[s]);
                    } else {
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            tma_load_2d(kt + c * 8192, &tmK, 64 * c, y, &full[s]);
                            tma_load_2d(kt + C::TILE + c * 8192, &tmV, 64 * c, y, &full[s]);
                        }
                    }
                }
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
                ++used;
                advance();
            }
        };
        tree_entries<false>(p, pos, end, tile, unit, true, ok, issue);
        // every copy lands before the block ends, also when a consumer gave up (earlier uses of a stage
        // were complete before it was filled again)
        if (lane == 0) {
            for (int i = 0; i < p.nk && i < used; ++i) {
                s = s == 0 ? p.nk - 1 : s - 1;
                if (s == p.nk - 1) par ^= 1u;
                if (!mbar_wait(&full[s], par, p.status, kTreeDetail | 0x14u)) break;
            }
            if (drafts > 0) mbar_wait(&dfull, dpar ^ 1u, p.status, kTreeDetail | 0x15u);
        }
        __syncthreads();
        return;
    }

    // ---------------------------------------------------- consumers
    const int r = lane >> 2, q4 = lane & 3, mi = lane >> 3, mr = lane & 7;
    const int key0 = 16 * warp;         // this warp's keys of a unit
    while (pos < end) {
        const int b = static_cast<int>(tile / p.rows_per_seq);
        const int rem = static_cast<int>(tile % p.rows_per_seq);
        const int hs = rem / p.mt, base = (rem % p.mt) * p.rpt;  // the row tile's rows base .. of the selection row's
        const int rows = min(p.rpt, p.gh * p.T - base);
        const int units = tree_units(p, tree_len(p, b));
        const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
        const int64_t out0 = (static_cast<int64_t>(b) * p.Hq + hs * p.gh) * p.T + base;  // first output row

        FewState<D, E4M3, NT> st;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) st.o[t][j][0] = st.o[t][j][1] = st.o[t][j][2] = st.o[t][j][3] = 0.f;
            st.ref[t][0] = st.ref[t][1] = kTreeNone;
            st.l[t][0] = st.l[t][1] = 0.f;
            if constexpr (E4M3) st.f[t][0] = st.f[t][1] = 1.f;
        }
        st.emax = 0;
        st.fresh = true;

        // Q as the B operand: row 8 t + r; bf16: dims 16 k + 2 q4 (+ 8); e4m3: dims 16 k + 4 q4 .. + 3 as
        // fp16, scaled; and the score factors of this thread's rows 8 t + 2 q4, + 1
        uint32_t qf[NT][D / 16][2];
        float f[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const __nv_bfloat16* q = p.Q + (out0 + 8 * t + r) * D;
            const bool have = 8 * t + r < rows;
            if constexpr (E4M3) {
                uint2 x[D / 16];
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    x[k] = have ? __ldg(reinterpret_cast<const uint2*>(q + 16 * k) + q4) : make_uint2(0u, 0u);
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[k].x << 16)), fabsf(__uint_as_float(x[k].x & 0xFFFF0000u))));
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[k].y << 16)), fabsf(__uint_as_float(x[k].y & 0xFFFF0000u))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // exponent field of the factor that brings the maximum to [2^14, 2^15)
                const int e = min(253, 268 - static_cast<int>(__float_as_uint(top) >> 23));
                const float g = __uint_as_float(static_cast<uint32_t>(e) << 23);
                const float back = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qf[t][k][0] = pack_f16x2(__uint_as_float(x[k].x << 16) * g, __uint_as_float(x[k].x & 0xFFFF0000u) * g);
                    qf[t][k][1] = pack_f16x2(__uint_as_float(x[k].y << 16) * g, __uint_as_float(x[k].y & 0xFFFF0000u) * g);
                }
                f[t][0] = __shfl_sync(0xFFFFFFFFu, back, 8 * q4);       // row 2 q4 lives in lanes 8 q4 ..
                f[t][1] = __shfl_sync(0xFFFFFFFFu, back, 8 * q4 + 4);
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(q + 16 * k) + q4;
                    qf[t][k][0] = have ? __ldg(w) : 0u;
                    qf[t][k][1] = have ? __ldg(w + 4) : 0u;
                }
                f[t][0] = f[t][1] = p.scale_log2;
            }
        }

        while (ok) {
            ok = mbar_wait(&full[s], par, p.status, kTreeDetail | 0x16u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const int lim = meta[s];
            if (lim == 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
                advance();
                break;
            }
            uint8_t* kt = ring + s * C::STAGE;
            uint8_t* es = exps + s * 128;
            const uint32_t kb = smem_u32(kt), vb = kb + C::TILE;
            if (key0 < lim) {
                if (key0 + 16 > lim) {
                    // rows past the sequence hold whatever the cache held: V's must not reach the product
                    // as NaN (0 * NaN), nor V's exponents
                    for (int e = lane; e < 16 * (C::ROW / 16); e += 32) {
                        const int key = key0 + e / (C::ROW / 16), c = e % (C::ROW / 16);
                        if (key >= lim) {
                            const uint32_t o = E4M3 ? few_at_e4m3<D>(key, c) : (c / 8) * 8192 + few_at128(key, c % 8);
                            *reinterpret_cast<uint4*>(kt + C::TILE + o) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (E4M3 && lane < 16 && key0 + lane >= lim) es[key0 + lane] = es[64 + key0 + lane] = 0;
                    __syncwarp();
                }
                float x[NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
                if constexpr (E4M3) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t a[4];  // (keys 0-7, chunk 2c), (keys 8-15, 2c), (keys 0-7, 2c + 1), (keys 8-15, 2c + 1)
                        few_ldsm4(kb + few_at_e4m3<D>(key0 + mr + 8 * (mi & 1), 2 * c + (mi >> 1)), a);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a0 = e4m3x2_f16x2<false>(a[2 * h]), a2 = e4m3x2_f16x2<true>(a[2 * h]);
                            const uint32_t a1 = e4m3x2_f16x2<false>(a[2 * h + 1]), a3 = e4m3x2_f16x2<true>(a[2 * h + 1]);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                few_mma<true>(x[t], a0, a1, a2, a3, qf[t][2 * c + h][0], qf[t][2 * c + h][1]);
                        }
                    }
                    const float k0 = __uint_as_float(static_cast<uint32_t>(es[key0 + r]) << 23);
                    const float k1 = __uint_as_float(static_cast<uint32_t>(es[key0 + r + 8]) << 23);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        x[t][0] *= k0 * f[t][0];
                        x[t][1] *= k0 * f[t][1];
                        x[t][2] *= k1 * f[t][0];
                        x[t][3] *= k1 * f[t][1];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t a[4];
                        few_ldsm4(kb + (k / 4) * 8192 + few_at128(key0 + mr + 8 * (mi & 1), 2 * (k % 4) + (mi >> 1)), a);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            few_mma<false>(x[t], a[0], a[1], a[2], a[3], qf[t][k][0], qf[t][k][1]);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[t][e] *= p.scale_log2;
                    }
                }
                if (key0 + 16 > lim) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (key0 + r >= lim) x[t][0] = x[t][1] = -INFINITY;
                        if (key0 + r + 8 >= lim) x[t][2] = x[t][3] = -INFINITY;
                    }
                }
                few_softmax<D, E4M3, NT, false>(st, x, E4M3 ? es[64 + key0 + r] : 0, E4M3 ? es[64 + key0 + r + 8] : 0, 0.f, 0.f);
                uint32_t pb[NT][2];  // P^T: keys 2 q4, + 1 (+ 8) of row 8 t + r
                if constexpr (E4M3) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        pb[t][0] = few_transpose(pack_f16x2(x[t][0], x[t][1]));
                        pb[t][1] = few_transpose(pack_f16x2(x[t][2], x[t][3]));
                    }
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t a[4];  // (keys 0-7, chunk 2c), (keys 8-15, 2c), (keys 0-7, 2c + 1), (keys 8-15, 2c + 1)
                        few_ldsm4_t(vb + few_at_e4m3<D>(key0 + mr + 8 * (mi & 1), 2 * c + (mi >> 1)), a);
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[i] = __byte_perm(a[i], 0u, 0x3120);  // (even, even, odd, odd)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a0 = e4m3x2_f16x2<false>(a[2 * h]), a1 = e4m3x2_f16x2<true>(a[2 * h]);
                            const uint32_t a2 = e4m3x2_f16x2<false>(a[2 * h + 1]), a3 = e4m3x2_f16x2<true>(a[2 * h + 1]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) few_mma<true>(st.o[t][2 * c + h], a0, a1, a2, a3, pb[t][0], pb[t][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        pb[t][0] = few_transpose(pack_bf16x2(x[t][0], x[t][1]));
                        pb[t][1] = few_transpose(pack_bf16x2(x[t][2], x[t][3]));
                    }
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t a[4];
                        few_ldsm4_t(vb + (j / 4) * 8192 + few_at128(key0 + mr + 8 * (mi >> 1), 2 * (j % 4) + (mi & 1)), a);
#pragma unroll
                        for (int t = 0; t < NT; ++t) few_mma<false>(st.o[t][j], a[0], a[1], a[2], a[3], pb[t][0], pb[t][1]);
                    }
                }
                if (key0 + 16 > lim) fence_proxy_async_smem();  // the zeros, before the next copy into the stage
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            advance();
        }

        if (u1 == units) {
            // ---- the drafted tokens (16 at most): the first warp takes them
            if (ok) ok = mbar_wait(&dfull, dpar, p.status, kTreeDetail | 0x17u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
                dpar ^= 1u;
                if (warp == 0) {
                    const uint64_t live = (1ull << p.T) - 1ull;
                    uint32_t mk[NT][2];  // the ancestor bits of this thread's rows
                    float x[NT][4];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 8 * t + 2 * q4 + e;
                            mk[t][e] = row < rows ? static_cast<uint32_t>(__ldg(p.mask + static_cast<int64_t>(b) * p.T + (base + row) % p.T) & live) : 0u;
                        }
                        x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
                    }
                    const uint32_t kb = smem_u32(dk_s);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t a[4];
                        few_ldsm4(kb + (k / 4) * 2048 + few_at128(mr + 8 * (mi & 1), 2 * (k % 4) + (mi >> 1)), a);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            uint32_t b0, b1;
                            if constexpr (E4M3) {  // bf16 rows as they are
                                const uint32_t* w = reinterpret_cast<const uint32_t*>(p.Q + (out0 + 8 * t + r) * D + 16 * k) + q4;
                                const bool have = 8 * t + r < rows;
                                b0 = have ? __ldg(w) : 0u;
                                b1 = have ? __ldg(w + 4) : 0u;
                            } else {
                                b0 = qf[t][k][0];
                                b1 = qf[t][k][1];
                            }
                            few_mma<false>(x[t], a[0], a[1], a[2], a[3], b0, b1);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            x[t][e] = (mk[t][e] >> r) & 1u ? x[t][e] * p.scale_log2 : -INFINITY;
                            x[t][2 + e] = (mk[t][e] >> (r + 8)) & 1u ? x[t][2 + e] * p.scale_log2 : -INFINITY;
                        }
                    }
                    float ed0 = 0.f, ed1 = 0.f;  // of this thread's keys, the exponents that their values would have in the cache
                    if constexpr (E4M3) {
                        uint32_t top = 0;  // largest finite magnitude of key lane % 16, half of the dims a lane
                        if ((lane & 15) < p.T) {
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                const int c = (lane >> 4) * (D / 16) + i;
                                const uint4 v = *reinterpret_cast<const uint4*>(dk_s + C::DRAFT + (c / 8) * 2048 + few_at128(lane & 15, c % 8));
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
                                    top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                                }
                            }
                        }
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                        const float e = fmaxf(kFewDraftMin, static_cast<float>(static_cast<int>(top >> 7) - 127 - 8));
                        ed0 = __shfl_sync(0xFFFFFFFFu, e, r);
                        ed1 = __shfl_sync(0xFFFFFFFFu, e, r + 8);
                    }
                    few_softmax<D, E4M3, NT, true>(st, x, 0, 0, ed0, ed1);
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        pb[t][0] = few_transpose(pack_bf16x2(x[t][0], x[t][1]));
                        pb[t][1] = few_transpose(pack_bf16x2(x[t][2], x[t][3]));
                    }
                    // V value by value, in the order of O's tiles: rows past the tokens are left out, and so is a
                    // value that is not finite, which would reach every token through 0 * x
                    auto value = [&](int key, int dim) -> uint32_t {
                        if (key >= p.T) return 0u;
                        return *reinterpret_cast<const uint16_t*>(dk_s + C::DRAFT + (dim / 64) * 2048 +
                                                                  few_at128(key, (dim % 64) / 8) + 2 * (dim % 8));
                    };
                    auto finite = [](uint32_t h) { return (h & 0x7F80u) != 0x7F80u; };
                    bool odd = false;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        const int d0 = 16 * j + (E4M3 ? 2 * r : r), d1 = E4M3 ? d0 + 1 : d0 + 8;
                        uint32_t a[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int dim = i & 1 ? d1 : d0, key = 2 * q4 + 8 * (i >> 1);
                            uint32_t lo = value(key, dim), hi = value(key + 1, dim);
                            odd = odd || !finite(lo) || !finite(hi);
                            lo = finite(lo) ? lo : 0u;
                            hi = finite(hi) ? hi : 0u;
                            a[i] = lo | (hi << 16);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) few_mma<false>(st.o[t][j], a[0], a[1], a[2], a[3], pb[t][0], pb[t][1]);
                    }
                    if (__any_sync(0xFFFFFFFFu, odd)) {  // given to the tokens that attend it
                        for (int key = 0; key < p.T; ++key) {
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                const int d0 = 16 * j + (E4M3 ? 2 * r : r), d1 = E4M3 ? d0 + 1 : d0 + 8;
                                const uint32_t v0 = value(key, d0), v1 = value(key, d1);
#pragma unroll
                                for (int t = 0; t < NT; ++t) {
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        if (!((mk[t][e] >> key) & 1u)) continue;
                                        if (!finite(v0)) st.o[t][j][e] += __uint_as_float(v0 << 16);
                                        if (!finite(v1)) st.o[t][j][2 + e] += __uint_as_float(v1 << 16);
                                    }
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&dempty);
            }
        }

        // ---- the piece's end: the four warps meet in shared memory, CH dims at a time
        float uf[NT][2];  // O's unit
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = st.l[t][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
                if (r == 0) {
                    const int row = warp * C::RM + 8 * t + 2 * q4 + e;
                    cml[2 * row] = l == 0.f ? -INFINITY : st.ref[t][e];
                    cml[2 * row + 1] = l;
                }
                if constexpr (E4M3) uf[t][e] = __uint_as_float((254u << 23) - __float_as_uint(st.f[t][e]));  // 1 / f
                else uf[t][e] = 1.f;
            }
        }
        const bool whole = unit == 0 && u1 == units;
        // partial slots: 2c for a piece that goes on with a row tile, 2c + 1 for one that begins it
        float* part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (unit == 0 ? 1 : 0)) * C::RM * (D + 2);
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += C::CH) {
#pragma unroll
            for (int jj = 0; jj < C::CH / 16; ++jj) {
                const int j = c0 / 16 + jj;
                const int d0 = 16 * jj + (E4M3 ? 2 * r : r), d1 = E4M3 ? d0 + 1 : d0 + 8;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float* at = comb + (warp * C::RM + 8 * t + 2 * q4 + e) * C::CH;
                        at[d0] = st.o[t][j][e] * uf[t][e];
                        at[d1] = st.o[t][j][2 + e] * uf[t][e];
                    }
                }
            }
            named_bar_sync(1, 128);
            for (int e = tid; e < C::RM * C::CH; e += 128) {
                const int row = e / C::CH, d = c0 + e % C::CH;
                float M = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) M = fmaxf(M, cml[2 * (k * C::RM + row)]);
                float v = 0.f, l = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float mk = cml[2 * (k * C::RM + row)], lk = cml[2 * (k * C::RM + row) + 1];
                    const float w = mk == -INFINITY ? 0.f : fast_exp2(mk - M);  // a warp without a key for the row
                    v += w * comb[(k * C::RM + row) * C::CH + e % C::CH];
                    l += w * lk;
                }
                if (whole) {
                    if (row < rows) {
                        p.O[(out0 + row) * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : v / l);
                        if (d == 0 && p.lse != nullptr)
                            p.lse[out0 + row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
                    }
                } else {
                    part[row * D + d] = v;
                    if (d == 0) {
                        part[C::RM * D + 2 * row] = l == 0.f ? -INFINITY : M;
                        part[C::RM * D + 2 * row + 1] = l;
                    }
                }
            }
            named_bar_sync(1, 128);
        }
        pos += u1 - unit;
        unit = 0;
        ++tile;
    }
    __syncthreads();
}

template <int D, bool E4M3, int NT>
static bool launch_few(TreeParams p, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dk,
                       const CUtensorMap& dv, cudaStream_t st, int32_t* launches) {
    using C = FewCfg<D, E4M3, NT>;
    constexpr int budget = (C::CTAS == 3 ? 74 : 112) * 1024;  // of the SM's shared memory
    constexpr int fit = (budget - C::FIXED) / (C::STAGE + C::EXPS);
    static_assert(fit >= 2, "two stages must fit");
    p.nk = fit < kFewStages ? fit : kFewStages;
    p.nv = 0;
    const int smem = C::FIXED + p.nk * (C::STAGE + C::EXPS);
    static std::atomic<uint64_t> configured{0};
    if (!configure_smem_once(reinterpret_cast<const void*>(attn_tree_few_kernel<D, E4M3, NT>), smem, configured))
        return false;
    attn_tree_few_kernel<D, E4M3, NT><<<p.runs, kFewThreads, smem, st>>>(k, v, dk, dv, p);
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    return launch_tree_merge(p, D, C::RM, st, launches);
}

bool launch_attn_tree_few(TreeParams p, int D, bool e4m3, int rm, const void* K, const void* Kc, const void* Vc,
                          cudaStream_t st, int32_t* launches) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * p.cap, drows = static_cast<int64_t>(p.B) * p.Hkv * p.T;
    CUtensorMap k, v, dk, dv;
    if (!make_tmap_2d(&dk, K, drows, D, 16) || !make_tmap_2d(&dv, p.DV, drows, D, 16)) return false;
    if (e4m3 ? !make_tmap_2d_u8(&k, Kc, rows, D, 64) || !make_tmap_2d_u8(&v, Vc, rows, D, 64)
             : !make_tmap_2d(&k, Kc, rows, D, 64) || !make_tmap_2d(&v, Vc, rows, D, 64))
        return false;
#define PISA_FEW_CASE(DD, EE, NN) \
    if (D == DD && e4m3 == EE && rm == 8 * NN) return launch_few<DD, EE, NN>(p, k, v, dk, dv, st, launches);
    PISA_FEW_CASE(64, false, 1)
    PISA_FEW_CASE(64, false, 2)
    PISA_FEW_CASE(64, true, 1)
    PISA_FEW_CASE(64, true, 2)
    PISA_FEW_CASE(128, false, 1)
    PISA_FEW_CASE(128, false, 2)
    PISA_FEW_CASE(128, true, 1)
    PISA_FEW_CASE(128, true, 2)
#undef PISA_FEW_CASE
    return false;
}

}  // namespace pisa
