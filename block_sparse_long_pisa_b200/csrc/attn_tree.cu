// Attention of a tree of drafted tokens over a K/V cache (one drafted token is plain decode).
//
//   rows   the T drafted tokens of the gh query heads that share a selection row: gh * T rows, in
//          row tiles of RM = 16 MG, the M side of every product
//   keys   the drafted tokens themselves (masked by their ancestor bits), then the cache in units of
//          64 keys: selected blocks and tail, or all of it, up to the sequence's length
//   O = softmax(scale Q K^T) V with a running maximum and sum (fp32); no score leaves the registers
//
// Bound: with few rows, the bytes of the cache that are read (each byte once per row tile, and the
// row tiles of a sequence read it close together, from L2 after the first); with many rows the
// tensor cores.
//
// Work split. Sequences have unlike lengths that only the device knows, so the units of all row
// tiles are laid end to end and cut into equal runs, one per CTA of a fixed grid; a run may end one
// row tile, hold whole ones and begin another. A row tile inside one run is finished there; one that
// crosses runs leaves partial (o, m, l) that attn_tree_merge_kernel joins in run order. Every CTA
// finds its run by summing the lengths itself: no scheduling pass, no atomics, and the same inputs
// give the same bits.
//
// CTA: one producer warp keeps a ring of units in flight by TMA (K and V tiles of 64 keys, 128- or
// 64-byte swizzle, and the exponent bytes of an e4m3 cache); MG x KS consumer warps take 16 rows and
// every KS-th 16-key chunk each, with mma.sync m16n8k16 (few rows: the chunks are split so that four
// warps share 16 rows; many rows: each warp has its own). Drafted K/V have a buffer of their own.
//
// e4m3 rows are used as fp16: e4m3 values are exact there, and one conversion instruction makes two.
//   * Q is scaled by a power of two per row to a maximum in [2^14, 2^15) and rounded to fp16, which
//     keeps bf16's 8 bits for values down to 2^-29 of the row's largest.
//   * K's row exponent and Q's come back as an exact factor of the score, in fp32.
//   * V's row exponent goes into P: P' = p 2^(e - u), u the largest exponent so far less 7, O in
//     units of 2^u. P <= 2^8 (below), so P' <= 2^15 fits fp16; P' keeps its 11 bits down to 2^-21
//     of the largest row times the largest p, and a floor of 2^-31 below.
//   * A byte tile's fragments come by ldmatrix as pairs of bytes, so the order of dims inside a
//     16-dim chunk (Q.K^T, where any order will do) and of output columns (P.V: even dims in one
//     n-tile, odd in the next) is the one that needs no shuffling.
// P is bf16 for a bf16 cache (range of V) and for the drafted tokens.
//
// The running maximum moves only when a score exceeds it by 2^8, so O is rescaled rarely.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pisa_device.cuh"

namespace pisa {

constexpr uint32_t kTreeDetail = kKernTree << 8;
constexpr float kTreeLazy = 8.0f;   // log2 units a score may exceed the kept maximum by
constexpr int kTreeUMin = -100;     // smallest unit exponent of O (e4m3)

// ---------------------------------------------------------------- the runs

// Units of one row tile of sequence b: the drafted tokens, then the cache.
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

// ---------------------------------------------------------------- fragments

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two e4m3 values (low 16 bits) -> two fp16
__device__ __forceinline__ uint32_t f16_of(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(two));
    return h;
}
__device__ __forceinline__ uint32_t f16_of_hi(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(two));
    return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// byte offset of 16-byte chunk `c` of row `row` in a tile of 128-byte (64-byte) swizzled rows
__device__ __forceinline__ uint32_t at128(int row, int c) {
    return static_cast<uint32_t>(row * 128 + ((c ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint32_t at64(int row, int c) {
    return static_cast<uint32_t>(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ float pow2i(int e) {  // e in [-126, 127]
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Rows r and r + 8 of one warp: running maximum (log2 units), sum of this thread's columns, output
// accumulators, and the unit exponent of the output (e4m3).
template <int D>
struct TreeState {
    float o[D / 8][4];
    float m0, m1, l0, l1;
    int u;
    bool unit_set;
};

template <int D>
__device__ __forceinline__ void scale_rows(TreeState<D>& s, float a0, float a1) {
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
        s.o[j][0] *= a0;
        s.o[j][1] *= a0;
        s.o[j][2] *= a1;
        s.o[j][3] *= a1;
    }
}

// Scores (log2 units, -inf where masked) -> probabilities against the running maximum, which moves
// when a score exceeds it by kTreeLazy. NT n-tiles of 8 keys.
template <int D, int NT>
__device__ __forceinline__ void softmax_step(TreeState<D>& s, float (&sc)[NT][4]) {
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        x0 = fmax3(x0, sc[n][0], sc[n][1]);
        x1 = fmax3(x1, sc[n][2], sc[n][3]);
    }
    x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, 1));
    x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 2));
    x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, 2));
    const bool up0 = x0 > s.m0 + kTreeLazy, up1 = x1 > s.m1 + kTreeLazy;
    if (__any_sync(0xFFFFFFFFu, up0 || up1)) {
        const float a0 = up0 ? fast_exp2(s.m0 - x0) : 1.f, a1 = up1 ? fast_exp2(s.m1 - x1) : 1.f;
        s.m0 = up0 ? x0 : s.m0;
        s.m1 = up1 ? x1 : s.m1;
        s.l0 *= a0;
        s.l1 *= a1;
        scale_rows<D>(s, a0, a1);
    }
    // a row with no key yet keeps m = -inf: its scores are all -inf and give 0
    const float r0 = s.m0 == -INFINITY ? 0.f : s.m0, r1 = s.m1 == -INFINITY ? 0.f : s.m1;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        sc[n][0] = fast_exp2(sc[n][0] - r0);
        sc[n][1] = fast_exp2(sc[n][1] - r0);
        sc[n][2] = fast_exp2(sc[n][2] - r1);
        sc[n][3] = fast_exp2(sc[n][3] - r1);
        s.l0 += sc[n][0] + sc[n][1];
        s.l1 += sc[n][2] + sc[n][3];
    }
}

// Q.K^T of 16 keys from a bf16 tile (128-byte swizzled column tiles of 64 dims, SUB bytes apart).
template <int D>
__device__ __forceinline__ void scores_bf16(const uint32_t (&q)[D / 16][4], uint32_t kbase, int sub, int key0,
                                            float (&c0)[4], float (&c1)[4]) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        float (&c)[4] = nt == 0 ? c0 : c1;
        c[0] = c[1] = c[2] = c[3] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const int dim = 32 * j + 8 * mi;
            uint32_t b[4];
            ldsm4(kbase + (dim / 64) * sub + at128(key0 + 8 * nt + mr, (dim % 64) / 8), b);
            mma16816<false>(c, q[2 * j], b[0], b[1]);
            mma16816<false>(c, q[2 * j + 1], b[2], b[3]);
        }
    }
}
template <int D>
__device__ __forceinline__ void pv_bf16(TreeState<D>& s, const uint32_t (&p)[4], uint32_t vbase, int sub, int key0) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        const int dim = 16 * j + 8 * (mi >> 1);
        uint32_t b[4];
        ldsm4_t(vbase + (dim / 64) * sub + at128(key0 + mr + 8 * (mi & 1), (dim % 64) / 8), b);
        mma16816<false>(s.o[2 * j], p, b[0], b[1]);
        mma16816<false>(s.o[2 * j + 1], p, b[2], b[3]);
    }
}

template <int D>
__device__ __forceinline__ uint32_t at_e4m3(int key, int c) {
    return D == 128 ? at128(key, c) : at64(key, c);
}
// Q.K^T of 16 keys from an e4m3 tile; a thread's four bytes of a 16-dim chunk are dims 4 (lane % 4) ..
template <int D>
__device__ __forceinline__ void scores_e4m3(const uint32_t (&q)[D / 16][4], uint32_t kbase, int key0, float (&c0)[4],
                                            float (&c1)[4]) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        float (&c)[4] = nt == 0 ? c0 : c1;
        c[0] = c[1] = c[2] = c[3] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            uint32_t b[4];
            ldsm4(kbase + at_e4m3<D>(key0 + 8 * nt + mr, 4 * j + mi), b);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma16816<true>(c, q[4 * j + i], f16_of(b[i]), f16_of_hi(b[i]));
        }
    }
}
// P.V of 16 keys: n-tile 2g takes the even dims of 16-dim chunk g, n-tile 2g + 1 the odd ones.
template <int D>
__device__ __forceinline__ void pv_e4m3(TreeState<D>& s, const uint32_t (&p)[4], uint32_t vbase, int key0) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        uint32_t b[4];
        ldsm4_t(vbase + at_e4m3<D>(key0 + mr + 8 * (mi & 1), 2 * j + (mi >> 1)), b);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __byte_perm(b[i], 0u, 0x3120);  // (even, even, odd, odd)
        mma16816<true>(s.o[4 * j], p, f16_of(b[0]), f16_of(b[1]));
        mma16816<true>(s.o[4 * j + 1], p, f16_of_hi(b[0]), f16_of_hi(b[1]));
        mma16816<true>(s.o[4 * j + 2], p, f16_of(b[2]), f16_of(b[3]));
        mma16816<true>(s.o[4 * j + 3], p, f16_of_hi(b[2]), f16_of_hi(b[3]));
    }
}

// Output columns from the bf16 order (n-tile j: dims 8j + 2 (lane % 4), + 1) to the e4m3 order
// (n-tiles 2g, 2g + 1: dims 16g + 4 (lane % 4) + {0, 2} and + {1, 3}).
template <int D>
__device__ __forceinline__ void to_paired_columns(TreeState<D>& s) {
    const int lane = threadIdx.x & 31, q = lane & 3;
    const int a = (lane & ~3) | ((2 * q) & 3), b = (lane & ~3) | ((2 * q + 1) & 3);
#pragma unroll
    for (int g = 0; g < D / 16; ++g) {
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
            const float e0 = s.o[2 * g][r], e1 = s.o[2 * g][r + 1], f0 = s.o[2 * g + 1][r], f1 = s.o[2 * g + 1][r + 1];
            const float ea0 = __shfl_sync(0xFFFFFFFFu, e0, a), ea1 = __shfl_sync(0xFFFFFFFFu, e1, a);
            const float eb0 = __shfl_sync(0xFFFFFFFFu, e0, b), eb1 = __shfl_sync(0xFFFFFFFFu, e1, b);
            const float fa0 = __shfl_sync(0xFFFFFFFFu, f0, a), fa1 = __shfl_sync(0xFFFFFFFFu, f1, a);
            const float fb0 = __shfl_sync(0xFFFFFFFFu, f0, b), fb1 = __shfl_sync(0xFFFFFFFFu, f1, b);
            // dims 4q, 4q+1 live in lane 2q of the half tile (q < 2: first, else second), 4q+2, +3 in the next
            s.o[2 * g][r] = q < 2 ? ea0 : fa0;
            s.o[2 * g + 1][r] = q < 2 ? ea1 : fa1;
            s.o[2 * g][r + 1] = q < 2 ? eb0 : fb0;
            s.o[2 * g + 1][r + 1] = q < 2 ? eb1 : fb1;
        }
    }
}

// ---------------------------------------------------------------- the kernel

template <int D, bool E4M3>
struct TreeCfg {
    static constexpr int ROW = E4M3 ? D : 2 * D;           // bytes of a cache row
    static constexpr int TILE = 64 * ROW;                  // K (or V) of one unit
    static constexpr int EXPS = E4M3 ? 128 : 0;            // exponent bytes of K and of V
    static constexpr int STAGE = 2 * TILE;
};

// Bytes of dynamic shared memory: ring, exponents, drafted K/V (tp rows), and the combine area.
template <int D, bool E4M3, int MG, int KS>
constexpr size_t tree_smem(int nstg, int tp) {
    return 1024 + static_cast<size_t>(nstg) * (TreeCfg<D, E4M3>::STAGE + TreeCfg<D, E4M3>::EXPS) +
           2 * static_cast<size_t>(tp) * 2 * D + (KS > 1 ? static_cast<size_t>(KS) * 16 * MG * (16 + 2) * 4 : 0);
}

template <int D, bool E4M3, int MG, int KS>
__global__ void __launch_bounds__((MG * KS + 1) * 32, MG == 8 ? 1 : 2)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                     const TreeParams p) {
    using C = TreeCfg<D, E4M3>;
    constexpr int W = MG * KS;       // consumer warps
    constexpr int NCH = 4 / KS;      // 16-key chunks of a unit per warp
    constexpr int RM = 16 * MG;
    constexpr int kMaxStages = 8;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* dk_s = ring + p.nstg * C::STAGE;              // drafted K, then V: [D/64][tp][128 B]
    const int dsub = p.tp * 128, dtile = (D / 64) * dsub;
    uint8_t* exps = dk_s + 2 * dtile;                      // [stage][K 64, V 64]
    float* comb = reinterpret_cast<float*>(exps + p.nstg * C::EXPS);
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], dfull, dempty;
    __shared__ int meta[kMaxStages];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const TreeJob job = tree_job(p);
    if (static_cast<int64_t>(blockIdx.x) >= job.runs) return;
    int64_t pos = job.begin(blockIdx.x);
    const int64_t end = job.begin(blockIdx.x + 1);
    int64_t tile;
    int unit;
    tree_find(p, pos, tile, unit);
    if (tid == 0) {
        for (int s = 0; s < p.nstg; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], W);
        }
        mbar_init(&dfull, 1);
        mbar_init(&dempty, W);
        fence_barrier_init();
    }
    __syncthreads();

    int s = 0;            // ring stage, and the parity of its current use
    uint32_t par = 0, dpar = 0;
    bool ok = true;       // cleared by a wait that ran out: nothing more is waited for
    auto advance = [&]() {
        if (++s == p.nstg) {
            s = 0;
            par ^= 1u;
        }
    };

    if (warp == W) {
        // ------------------------------------------------ producer
        int used = 0, drafts = 0;   // ring slots and draft buffers handed out (lane 0's copies: all full by the end)
        if (lane == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            prefetch_tmap(&tmDK);
            prefetch_tmap(&tmDV);
        }
        while (pos < end && ok) {
            const int b = static_cast<int>(tile / p.rows_per_seq);
            const int hs = static_cast<int>(tile % p.rows_per_seq) / p.mt;
            const int kvh = p.per_qhead ? hs / p.g : hs;
            const int64_t plane = static_cast<int64_t>(b) * p.Hkv + kvh;
            const int len = tree_len(p, b);
            const int units = tree_units(p, len);
            const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
            const bool first_of_seq = tile % p.rows_per_seq == 0 && unit == 0;
            if (first_of_seq && lane == 0 && p.len[b] != len)
                record_error(p.status, PISA_ERR_BAD_INDEX, kTreeDetail | 0xB0u);
            int u = unit;
            if (u == 0) {
                if (lane == 0) {
                    ok = drafts == 0 || mbar_wait(&dempty, dpar ^ 1u, p.status, kTreeDetail | 0x01u);
                    if (ok) {
                        mbar_arrive_expect_tx(&dfull, 2 * dtile);
                        const int y = static_cast<int>(plane * p.T);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            tma_load_2d(dk_s + c * dsub, &tmDK, 64 * c, y, &dfull);
                            tma_load_2d(dk_s + dtile + c * dsub, &tmDV, 64 * c, y, &dfull);
                        }
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (ok) {
                    ++drafts;
                    dpar ^= 1u;
                }
                ++u;
            }
            const int32_t* row = p.topk > 0 ? p.idx + (static_cast<int64_t>(b) * p.Hsel + hs) * p.topk : nullptr;
            const int nsel = p.topk * p.upb;
            while (u < u1 && ok) {
                // up to 32 units at a time: position of each unit's first key, -1 = nothing there
                const int n = min(32, u1 - u);
                int at = -1;
                if (lane < n) {
                    const int c = u + lane - 1;
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
                const uint32_t have = __ballot_sync(0xFFFFFFFFu, at >= 0 && at < len);
                for (uint32_t left = have; left != 0 && ok; left &= left - 1) {
                    const int a = __shfl_sync(0xFFFFFFFFu, at, __ffs(left) - 1);
                    if (lane == 0) {
                        ok = used < p.nstg || mbar_wait(&empty[s], par ^ 1u, p.status, kTreeDetail | 0x02u);
                        if (ok) {
                            meta[s] = min(64, len - a);
                            uint8_t* kt = ring + s * C::STAGE;
                            mbar_arrive_expect_tx(&full[s], C::STAGE + C::EXPS);
                            const int y = static_cast<int>(plane * p.cap + a);
                            if constexpr (E4M3) {
                                tma_load_2d(kt, &tmK, 0, y, &full[s]);
                                tma_load_2d(kt + C::TILE, &tmV, 0, y, &full[s]);
                                bulk_load(exps + s * 128, p.k_exp + plane * p.cap + a, 64, &full[s]);
                                bulk_load(exps + s * 128 + 64, p.v_exp + plane * p.cap + a, 64, &full[s]);
                            } else {
#pragma unroll
                                for (int c = 0; c < D / 64; ++c) {
                                    tma_load_2d(kt + c * 8192, &tmK, 64 * c, y, &full[s]);
                                    tma_load_2d(kt + C::TILE + c * 8192, &tmV, 64 * c, y, &full[s]);
                                }
                            }
                        }
                    }
                    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                    if (ok) {
                        ++used;
                        advance();
                    }
                }
                u += n;
            }
            // end of the piece: a slot without a tile
            if (ok) {
                if (lane == 0) {
                    ok = used < p.nstg || mbar_wait(&empty[s], par ^ 1u, p.status, kTreeDetail | 0x03u);
                    if (ok) {
                        meta[s] = 0;
                        mbar_arrive(&full[s]);
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (ok) {
                    ++used;
                    advance();
                }
            }
            pos += u1 - unit;
            unit = 0;
            ++tile;
        }
        // every copy lands before the block ends, also when a consumer gave up (a stage is always
        // waited for by its latest use; earlier uses were complete before it was filled again)
        if (lane == 0) {
            for (int i = 0; i < p.nstg && i < used; ++i) {
                s = s == 0 ? p.nstg - 1 : s - 1;
                if (s == p.nstg - 1) par ^= 1u;
                if (!mbar_wait(&full[s], par, p.status, kTreeDetail | 0x04u)) break;
            }
            if (drafts > 0) mbar_wait(&dfull, dpar ^ 1u, p.status, kTreeDetail | 0x05u);
        }
        __syncthreads();
        return;
    }

    // ---------------------------------------------------- consumers
    const int mg = warp % MG, kg = warp / MG;
    const int r = lane >> 2, q4 = lane & 3;
    const int rows = p.gh * p.T;
    while (pos < end) {
        const int b = static_cast<int>(tile / p.rows_per_seq);
        const int rem = static_cast<int>(tile % p.rows_per_seq);
        const int hs = rem / p.mt, row_base = (rem % p.mt) * RM;
        const int units = tree_units(p, tree_len(p, b));
        const int u1 = static_cast<int>(min(static_cast<int64_t>(units), unit + (end - pos)));
        const int64_t out0 = (static_cast<int64_t>(b) * p.Hq + hs * p.gh) * p.T;  // first output row of the group
        const int ra = row_base + 16 * mg + r, rb = ra + 8;                       // this thread's rows of the group
        const __nv_bfloat16* qa = p.Q + (out0 + ra) * D;
        const __nv_bfloat16* qb = p.Q + (out0 + rb) * D;

        TreeState<D> st;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) st.o[j][0] = st.o[j][1] = st.o[j][2] = st.o[j][3] = 0.f;
        st.m0 = st.m1 = -INFINITY;
        st.l0 = st.l1 = 0.f;
        st.u = 0;
        st.unit_set = false;

        uint32_t qf[D / 16][4];
        if (!E4M3 || unit == 0) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t* x = reinterpret_cast<const uint32_t*>(qa + 16 * k) + q4;
                const uint32_t* y = reinterpret_cast<const uint32_t*>(qb + 16 * k) + q4;
                qf[k][0] = ra < rows ? __ldg(x) : 0u;
                qf[k][1] = rb < rows ? __ldg(y) : 0u;
                qf[k][2] = ra < rows ? __ldg(x + 4) : 0u;
                qf[k][3] = rb < rows ? __ldg(y + 4) : 0u;
            }
        }
        if (unit == 0) {
            const uint64_t* mrow = p.mask + static_cast<int64_t>(b) * p.T;
            const uint64_t live = p.T == 64 ? ~0ull : (1ull << p.T) - 1ull;
            const uint64_t ma = ra < rows ? __ldg(mrow + ra % p.T) & live : 0ull;
            const uint64_t mb = rb < rows ? __ldg(mrow + rb % p.T) & live : 0ull;
            if (ok) ok = mbar_wait(&dfull, dpar, p.status, kTreeDetail | 0x06u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
                dpar ^= 1u;
                const uint32_t kb = smem_u32(dk_s), vb = kb + dtile;
                for (int c = kg; 16 * c < p.T; c += KS) {
                    const int key0 = 16 * c;
                    float sc[2][4];
                    scores_bf16<D>(qf, kb, dsub, key0, sc[0], sc[1]);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = key0 + 8 * n + 2 * q4 + e;
                            sc[n][e] = (ma >> key) & 1ull ? sc[n][e] * p.scale_log2 : -INFINITY;
                            sc[n][2 + e] = (mb >> key) & 1ull ? sc[n][2 + e] * p.scale_log2 : -INFINITY;
                        }
                    }
                    softmax_step<D, 2>(st, sc);
                    // an infinity or NaN among the chunk's values would reach masked rows through 0 * x
                    const int vr = key0 + (lane & 15);
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int ch = (lane >> 4) * (D / 16) + i;  // 16-byte chunk of the row
                        const uint4 x = *reinterpret_cast<const uint4*>(dk_s + dtile + (ch / 8) * dsub + at128(vr, ch % 8));
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                                     __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
                    }
                    const bool odd = max(top & 0xFFFFu, top >> 16) >= 0x7F80u;
                    if (!__any_sync(0xFFFFFFFFu, odd)) {
                        const uint32_t pa[4] = {pack_bf16x2(sc[0][0], sc[0][1]), pack_bf16x2(sc[0][2], sc[0][3]),
                                                pack_bf16x2(sc[1][0], sc[1][1]), pack_bf16x2(sc[1][2], sc[1][3])};
                        pv_bf16<D>(st, pa, vb, dsub, key0);
                    } else {
                        // key by key, attended keys only
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                for (int q = 0; q < 4; ++q) {
                                    const int key = key0 + 8 * n + 2 * q + e;
                                    const float pr = __shfl_sync(0xFFFFFFFFu, sc[n][e], (lane & ~3) | q);
                                    const float ps = __shfl_sync(0xFFFFFFFFu, sc[n][2 + e], (lane & ~3) | q);
                                    const bool ua = (ma >> key) & 1ull, ub = (mb >> key) & 1ull;
#pragma unroll
                                    for (int j = 0; j < D / 8; ++j) {
                                        const uint32_t x = *reinterpret_cast<const uint32_t*>(
                                            dk_s + dtile + (j / 8) * dsub + at128(key, j % 8) + 4 * q4);
                                        const float lo = __uint_as_float(x << 16), hi = __uint_as_float(x & 0xFFFF0000u);
                                        if (ua) {
                                            st.o[j][0] = fmaf(pr, lo, st.o[j][0]);
                                            st.o[j][1] = fmaf(pr, hi, st.o[j][1]);
                                        }
                                        if (ub) {
                                            st.o[j][2] = fmaf(ps, lo, st.o[j][2]);
                                            st.o[j][3] = fmaf(ps, hi, st.o[j][3]);
                                        }
                                    }
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&dempty);
                if constexpr (E4M3) to_paired_columns<D>(st);
            }
        }

        // e4m3: the rows of Q as fp16 at a power-of-two scale, dims in the order of the byte tiles
        float fa = p.scale_log2, fb = p.scale_log2;
        if constexpr (E4M3) {
            float ta = 0.f, tb = 0.f;
            uint2 xa[D / 16], xb[D / 16];
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                xa[k] = ra < rows ? __ldg(reinterpret_cast<const uint2*>(qa + 16 * k) + q4) : make_uint2(0u, 0u);
                xb[k] = rb < rows ? __ldg(reinterpret_cast<const uint2*>(qb + 16 * k) + q4) : make_uint2(0u, 0u);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t wa = i == 0 ? xa[k].x : xa[k].y, wb = i == 0 ? xb[k].x : xb[k].y;
                    ta = fmaxf(ta, fmaxf(fabsf(__uint_as_float(wa << 16)), fabsf(__uint_as_float(wa & 0xFFFF0000u))));
                    tb = fmaxf(tb, fmaxf(fabsf(__uint_as_float(wb << 16)), fabsf(__uint_as_float(wb & 0xFFFF0000u))));
                }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                ta = fmaxf(ta, __shfl_xor_sync(0xFFFFFFFFu, ta, o));
                tb = fmaxf(tb, __shfl_xor_sync(0xFFFFFFFFu, tb, o));
            }
            // exponent field of the factor that brings the maximum to [2^14, 2^15)
            const int ea = min(253, 268 - static_cast<int>(__float_as_uint(ta) >> 23));
            const int eb = min(253, 268 - static_cast<int>(__float_as_uint(tb) >> 23));
            const float ga = __uint_as_float(static_cast<uint32_t>(ea) << 23);
            const float gb = __uint_as_float(static_cast<uint32_t>(eb) << 23);
            fa *= __uint_as_float(static_cast<uint32_t>(254 - ea) << 23);
            fb *= __uint_as_float(static_cast<uint32_t>(254 - eb) << 23);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][0] = pack_f16x2(__uint_as_float(xa[k].x << 16) * ga, __uint_as_float(xa[k].x & 0xFFFF0000u) * ga);
                qf[k][1] = pack_f16x2(__uint_as_float(xb[k].x << 16) * gb, __uint_as_float(xb[k].x & 0xFFFF0000u) * gb);
                qf[k][2] = pack_f16x2(__uint_as_float(xa[k].y << 16) * ga, __uint_as_float(xa[k].y & 0xFFFF0000u) * ga);
                qf[k][3] = pack_f16x2(__uint_as_float(xb[k].y << 16) * gb, __uint_as_float(xb[k].y & 0xFFFF0000u) * gb);
            }
        }

        while (ok) {
            ok = mbar_wait(&full[s], par, p.status, kTreeDetail | 0x07u);
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
            if (lim < 64) {
                // rows past the sequence hold whatever the cache held: V's must not reach the product as
                // NaN (0 * NaN), exponents must not set the unit. Warps that share rows write the same 0s.
                for (int i = 0; i < NCH; ++i) {
                    const int key0 = 16 * (kg + i * KS);
                    for (int e = lane; e < 16 * (C::ROW / 16); e += 32) {
                        const int key = key0 + e / (C::ROW / 16), c = e % (C::ROW / 16);
                        if (key >= lim) {
                            const uint32_t o = E4M3 ? at_e4m3<D>(key, c) : (c / 8) * 8192 + at128(key, c % 8);
                            *reinterpret_cast<uint4*>(kt + C::TILE + o) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (E4M3 && lane < 16 && key0 + lane >= lim) es[key0 + lane] = es[64 + key0 + lane] = 0;
                }
                __syncwarp();
            }
            float sc[2 * NCH][4];
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int key0 = 16 * (kg + i * KS);
                if constexpr (E4M3) {
                    scores_e4m3<D>(qf, kb, key0, sc[2 * i], sc[2 * i + 1]);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint32_t two = *reinterpret_cast<const uint16_t*>(es + key0 + 8 * n + 2 * q4);
                        const float f0 = __uint_as_float((two & 0xFFu) << 23), f1 = __uint_as_float((two >> 8) << 23);
                        sc[2 * i + n][0] *= f0 * fa;
                        sc[2 * i + n][1] *= f1 * fa;
                        sc[2 * i + n][2] *= f0 * fb;
                        sc[2 * i + n][3] *= f1 * fb;
                    }
                } else {
                    scores_bf16<D>(qf, kb, 8192, key0, sc[2 * i], sc[2 * i + 1]);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[2 * i + n][e] *= p.scale_log2;
                    }
                }
                if (lim < 64) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int key = key0 + 8 * n + 2 * q4;
                        if (key >= lim) sc[2 * i + n][0] = sc[2 * i + n][2] = -INFINITY;
                        if (key + 1 >= lim) sc[2 * i + n][1] = sc[2 * i + n][3] = -INFINITY;
                    }
                }
            }
            if constexpr (E4M3) {
                // the unit exponent: the largest V exponent of this warp's keys so far, less 7
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4*>(es + 64 + 16 * (kg + i * KS));
                    top = __vmaxu4(top, __vmaxu4(__vmaxu4(x.x, x.y), __vmaxu4(x.z, x.w)));
                }
                top = __vmaxu4(top, top >> 16);
                top = max(top & 0xFFu, (top >> 8) & 0xFFu);
                const int u = max(kTreeUMin, min(static_cast<int>(top), 254) - 127 - 7);
                if (!st.unit_set || u > st.u) {
                    const float f = pow2i(max(-126, st.u - u));
                    scale_rows<D>(st, f, f);
                    st.u = u;
                    st.unit_set = true;
                }
            }
            softmax_step<D, 2 * NCH>(st, sc);
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int key0 = 16 * (kg + i * KS);
                uint32_t pa[4];
                if constexpr (E4M3) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint32_t two = *reinterpret_cast<const uint16_t*>(es + 64 + key0 + 8 * n + 2 * q4);
                        const int e0 = static_cast<int>(two & 0xFFu), e1 = static_cast<int>(two >> 8);
                        // a row of exponent 255 keeps its infinity: it is NaN for every token
                        const float f0 = __uint_as_float(static_cast<uint32_t>(e0 == 255 ? 255 : max(e0 - st.u, 0)) << 23);
                        const float f1 = __uint_as_float(static_cast<uint32_t>(e1 == 255 ? 255 : max(e1 - st.u, 0)) << 23);
                        pa[2 * n] = pack_f16x2(sc[2 * i + n][0] * f0, sc[2 * i + n][1] * f1);
                        pa[2 * n + 1] = pack_f16x2(sc[2 * i + n][2] * f0, sc[2 * i + n][3] * f1);
                    }
                    pv_e4m3<D>(st, pa, vb, key0);
                } else {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        pa[2 * n] = pack_bf16x2(sc[2 * i + n][0], sc[2 * i + n][1]);
                        pa[2 * n + 1] = pack_bf16x2(sc[2 * i + n][2], sc[2 * i + n][3]);
                    }
                    pv_bf16<D>(st, pa, vb, 8192, key0);
                }
            }
            if (lim < 64) fence_proxy_async_smem();  // this warp's zeros, before the next copy into the stage
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            advance();
        }

        // ---- the piece's end
        if constexpr (E4M3) {
            if (st.unit_set) {
                const float f = pow2i(st.u);
                scale_rows<D>(st, f, f);
            }
        }
        float l0 = st.l0, l1 = st.l1;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, o);
            l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, o);
        }
        const bool whole = unit == 0 && u1 == units;
        // partial slots: 2c for a piece that goes on with a row tile, 2c + 1 for one that begins it
        float* part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (unit == 0 ? 1 : 0)) * RM * (D + 2);
        // dims of accumulator element (j, e) of a row
        auto dim_of = [&](int j, int e) {
            return E4M3 ? 16 * (j / 2) + 4 * q4 + 2 * e + (j & 1) : 8 * j + 2 * q4 + e;
        };
        if constexpr (KS == 1) {
            const int la = 16 * mg + r, lb = la + 8;
            if (whole) {
                const float ia = l0 > 0.f || l0 != l0 ? 1.f / l0 : 0.f, ib = l1 > 0.f || l1 != l1 ? 1.f / l1 : 0.f;
#pragma unroll
                for (int g = 0; g < D / 16; ++g) {
                    if constexpr (E4M3) {
                        const int d = 16 * g + 4 * q4;
                        if (ra < rows)
                            *reinterpret_cast<uint2*>(p.O + (out0 + ra) * D + d) =
                                make_uint2(pack_bf16x2(st.o[2 * g][0] * ia, st.o[2 * g + 1][0] * ia),
                                           pack_bf16x2(st.o[2 * g][1] * ia, st.o[2 * g + 1][1] * ia));
                        if (rb < rows)
                            *reinterpret_cast<uint2*>(p.O + (out0 + rb) * D + d) =
                                make_uint2(pack_bf16x2(st.o[2 * g][2] * ib, st.o[2 * g + 1][2] * ib),
                                           pack_bf16x2(st.o[2 * g][3] * ib, st.o[2 * g + 1][3] * ib));
                    } else {
#pragma unroll
                        for (int j = 2 * g; j < 2 * g + 2; ++j) {
                            const int d = 8 * j + 2 * q4;
                            if (ra < rows)
                                *reinterpret_cast<uint32_t*>(p.O + (out0 + ra) * D + d) =
                                    pack_bf16x2(st.o[j][0] * ia, st.o[j][1] * ia);
                            if (rb < rows)
                                *reinterpret_cast<uint32_t*>(p.O + (out0 + rb) * D + d) =
                                    pack_bf16x2(st.o[j][2] * ib, st.o[j][3] * ib);
                        }
                    }
                }
                if (p.lse != nullptr && q4 == 0) {
                    if (ra < rows)
                        p.lse[out0 + ra] = l0 == 0.f ? -INFINITY : (st.m0 + log2f(l0)) * 0.69314718055994531f;
                    if (rb < rows)
                        p.lse[out0 + rb] = l1 == 0.f ? -INFINITY : (st.m1 + log2f(l1)) * 0.69314718055994531f;
                }
            } else {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        part[la * D + dim_of(j, e)] = st.o[j][e];
                        part[lb * D + dim_of(j, e)] = st.o[j][2 + e];
                    }
                }
                if (q4 == 0) {
                    part[RM * D + 2 * la] = st.m0;
                    part[RM * D + 2 * la + 1] = l0;
                    part[RM * D + 2 * lb] = st.m1;
                    part[RM * D + 2 * lb + 1] = l1;
                }
            }
        } else {
            // the KS warps of a row group meet in shared memory, 16 dims at a time
            float* cml = comb + KS * RM * 16;   // [kg][row][m, l]
            const int la = 16 * mg + r, lb = la + 8;
            if (q4 == 0) {
                cml[(kg * RM + la) * 2] = st.m0;
                cml[(kg * RM + la) * 2 + 1] = l0;
                cml[(kg * RM + lb) * 2] = st.m1;
                cml[(kg * RM + lb) * 2 + 1] = l1;
            }
            for (int g = 0; g < D / 16; ++g) {
#pragma unroll
                for (int gg = 0; gg < D / 16; ++gg) {
                    if (gg != g) continue;  // constant accumulator indices
#pragma unroll
                    for (int j = 2 * gg; j < 2 * gg + 2; ++j) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            comb[(kg * RM + la) * 16 + dim_of(j, e) - 16 * gg] = st.o[j][e];
                            comb[(kg * RM + lb) * 16 + dim_of(j, e) - 16 * gg] = st.o[j][2 + e];
                        }
                    }
                }
                named_bar_sync(1, W * 32);
                for (int e = tid; e < RM * 16; e += W * 32) {
                    const int row = e / 16, d = 16 * g + e % 16;
                    float M = -INFINITY;
#pragma unroll
                    for (int k = 0; k < KS; ++k) M = fmaxf(M, cml[(k * RM + row) * 2]);
                    float v = 0.f, l = 0.f;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const float mk = cml[(k * RM + row) * 2], lk = cml[(k * RM + row) * 2 + 1];
                        // a warp without a key for the row has l = 0 (and o = 0) unless it met a NaN
                        const float w = mk == -INFINITY ? (lk == 0.f ? 0.f : 1.f) : fast_exp2(mk - M);
                        v += w * comb[(k * RM + row) * 16 + e % 16];
                        l += w * lk;
                    }
                    const int rg = row_base + row;
                    if (whole) {
                        if (rg < rows) {
                            p.O[(out0 + rg) * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : v / l);
                            if (d == 0 && p.lse != nullptr)
                                p.lse[out0 + rg] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
                        }
                    } else {
                        part[row * D + d] = v;
                        if (d == 0) {
                            part[RM * D + 2 * row] = M;
                            part[RM * D + 2 * row + 1] = l;
                        }
                    }
                }
                named_bar_sync(1, W * 32);
            }
        }
        pos += u1 - unit;
        unit = 0;
        ++tile;
    }
    __syncthreads();
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

// Row tile of a group of `rows` rows: 16 rows (the chunks of a unit split over four warps), 32 (over
// two), 64 or 128; past 64 rows the size that pads least, the larger one on a tie.
int tree_row_tile(int rows) {
    if (rows <= 16) return 16;
    if (rows <= 32) return 32;
    if (rows <= 64) return 64;
    const int by64 = (rows + 63) / 64 * 64, by128 = (rows + 127) / 128 * 128;
    return by128 <= by64 ? 128 : 64;
}

template <int D, bool E4M3, int MG, int KS>
static bool launch_tree(TreeParams p, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dk,
                        const CUtensorMap& dv, cudaStream_t st, int32_t* launches) {
    using C = TreeCfg<D, E4M3>;
    // two CTAs share an SM's shared memory (one of 128 rows has it alone)
    const size_t budget = (MG == 8 ? 224 : 112) * 1024;
    int nstg = 8;
    while (nstg > 2 && tree_smem<D, E4M3, MG, KS>(nstg, p.tp) > budget) --nstg;
    p.nstg = nstg;
    const size_t smem = tree_smem<D, E4M3, MG, KS>(nstg, p.tp);
    static std::atomic<uint64_t> configured{0};
    if (!configure_smem_once(reinterpret_cast<const void*>(attn_tree_kernel<D, E4M3, MG, KS>), 227 * 1024 - 1024,
                             configured))
        return false;
    attn_tree_kernel<D, E4M3, MG, KS><<<p.runs, (MG * KS + 1) * 32, smem, st>>>(k, v, dk, dv, p);
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.rows_per_seq, 4 * MG);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, attn_tree_merge_kernel<D>, p, 16 * MG) != cudaSuccess) return false;
    ++*launches;
    return true;
}

template <int D, bool E4M3>
static bool launch_tree_rows(const TreeParams& p, int rm, const CUtensorMap& k, const CUtensorMap& v,
                             const CUtensorMap& dk, const CUtensorMap& dv, cudaStream_t st, int32_t* launches) {
    switch (rm) {
        case 16: return launch_tree<D, E4M3, 1, 4>(p, k, v, dk, dv, st, launches);
        case 32: return launch_tree<D, E4M3, 2, 2>(p, k, v, dk, dv, st, launches);
        case 64: return launch_tree<D, E4M3, 4, 1>(p, k, v, dk, dv, st, launches);
        default: return launch_tree<D, E4M3, 8, 1>(p, k, v, dk, dv, st, launches);
    }
}

bool launch_attn_tree(TreeParams p, int D, bool e4m3, int rm, const void* K, const void* V, const void* Kc,
                      const void* Vc, cudaStream_t st, int32_t* launches) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * p.cap, drows = static_cast<int64_t>(p.B) * p.Hkv * p.T;
    CUtensorMap k, v, dk, dv;
    if (!make_tmap_2d(&dk, K, drows, D, p.tp) || !make_tmap_2d(&dv, V, drows, D, p.tp)) return false;
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
