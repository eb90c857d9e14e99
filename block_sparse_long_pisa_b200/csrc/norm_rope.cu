// RMS norm of every query and key head and the rotation by position, in one pass over the packed
// projection, and its backward pass.
//
//   forward   r = (mean x^2 + eps)^(-1/2), u = x r w, y = R(pos) u
//   backward  du = R(pos)^T dy, dn = du w, dx = r (dn - x r^2 mean(dn x)), dw = sum du x r
//
// Both are bound by HBM: 2 bytes read and 2 written per value (forward), 4 read and 2 written
// (backward). What carries them:
//   * D/8 lanes hold one head row, 8 adjacent dims (16 bytes) each, so a row is one load and one
//     store per lane, and both reductions of a row are log2(D/8) shuffles. R is a multiple of 16,
//     so a lane's dims turn all or not at all, and its mates (i +- R/2) are one other lane's 8
//     dims: the raw bf16 words are exchanged (four shuffles), not the products.
//   * A group of lanes keeps one token and walks heads, so cos and sin stay in registers, folded
//     into the weights (y = r (x a + x_mate b) with a = w cos, b = -+ w_mate sin): one token's angles
//     are formed once, four per lane, and not once per head. The angle is pos * inv_freq in fp64, taken
//     modulo one turn before it is rounded to fp32: a far position keeps its phase (an fp32 product
//     is off by 2^-24 of an angle of 10^6, 0.06 rad).
//   * A tile is as many tokens as a block has lane groups: the tile's stores of one head are one
//     contiguous run (16 rows of 256 bytes at D = 128) although input and output orders differ.
//   * Few tokens (one decode step): tiles shrink to one token and its heads split over blocks, down
//     to one row per lane group, until the grid fills the SMs.
// The weight gradients are summed in registers along a block's tiles (a grid of at most
// kNormRopeBlocks blocks), then over the block's groups through shared memory, then over the blocks
// by a second kernel: fixed orders, no atomics.
//
// Measured (heads of 128, all dims turned): forward, 131,072 tokens of 32 + 8 heads, 2.68 GB in 464 us, 5.8 TB/s
// (88 % of the copy rate); 64 tokens of as many heads 5.2 us. Backward, 32,768 tokens of 16 + 16 heads, 0.81 GB in
// 166 us, 4.9 TB/s (74 %): rows travel through registers, and with the angles' products and the weight sums beside
// them two blocks fit an SM (128 registers and, D = 128, 52 bytes of spills a thread; at three blocks 584 bytes), so the
// loads in flight bound it (DRAM 54 %, issue 54 % in the profile). The forward pass spills 104 bytes at its three
// blocks. 3 x 1,537 tokens of 12 + 4 heads of 64: backward 20 us, 6 us of them the weight sums' kernel, which runs after
// the rows' one.
#include <cuda_bf16.h>

#include "pisa_device.cuh"

namespace pisa {

constexpr int kNrThreads = 256;

// 8 bf16 of a row as four packed fp32 pairs, and back (one rounding).
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = f2_pack(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        f2_unpack(f[k], lo, hi);
        w[k] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint64_t nr_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint4 load_row(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ uint4 shfl4(const uint4& v, int src) {
    return make_uint4(__shfl_sync(0xFFFFFFFFu, v.x, src), __shfl_sync(0xFFFFFFFFu, v.y, src),
                      __shfl_sync(0xFFFFFFFFu, v.z, src), __shfl_sync(0xFFFFFFFFu, v.w, src));
}

// Sum over the D/8 lanes of a row (every lane gets it).
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// What a lane needs to turn its 8 dims of one token: cos and the sine with the sign of its mate's
// share (forward), both 1 and 0 past the rotated dims.
struct Turn {
    float c[8], s[8];
};

// Where the lane's mates live. Half pairs: another lane; interleaved pairs: the lane itself.
template <int D>
struct LaneMap {
    int lane8;       // dim block of this lane: dims 8 lane8 ..
    int mate;        // warp lane whose words hold the mates (half pairs)
    bool turns, second;
    __device__ __forceinline__ LaneMap(int R, bool inter) {
        const int lane = threadIdx.x & 31;
        lane8 = lane % (D / 8);
        turns = 8 * lane8 < R;
        second = !inter && turns && 16 * lane8 >= R;
        const int d = inter || !turns ? 0 : (second ? -(R / 16) : R / 16);
        mate = lane + d;
    }
};

// cos and sin of a lane's dims at position pos. A lane forms four angles; with half pairs its mate
// needs the same eight and forms the other four.
template <int D, bool INTER>
__device__ __forceinline__ void form_turn(const NormRopeParams& p, const LaneMap<D>& lm, int64_t tok, Turn& t) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        t.c[k] = 1.f;
        t.s[k] = 0.f;
    }
    if (p.R == 0) return;
    const int i0 = INTER ? 4 * lm.lane8 : 8 * lm.lane8 - (lm.second ? p.R / 2 - 4 : 0);
    float c[4], s[4];
    if (lm.turns) {
        const double pos = static_cast<double>(__ldg(p.pos + tok));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const double turns = pos * static_cast<double>(__ldg(p.inv_freq + i0 + k)) * 0.15915494309189533577;
            sincospif(2.f * static_cast<float>(turns - rint(turns)), &s[k], &c[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = s[k] = 0.f;
    }
    if constexpr (INTER) {
        if (lm.turns) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                t.c[2 * k] = t.c[2 * k + 1] = c[k];
                t.s[2 * k] = -s[k];
                t.s[2 * k + 1] = s[k];
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float oc = __shfl_sync(0xFFFFFFFFu, c[k], lm.mate), os = __shfl_sync(0xFFFFFFFFu, s[k], lm.mate);
            if (lm.turns) {  // the first lane of the two formed the lower four
                t.c[k] = lm.second ? oc : c[k];
                t.c[4 + k] = lm.second ? c[k] : oc;
                t.s[k] = lm.second ? os : -s[k];
                t.s[4 + k] = lm.second ? s[k] : -os;
            }
        }
    }
}

// The mates' values of this lane's 8 dims: interleaved pairs are the lane's own, changed places.
template <bool INTER>
__device__ __forceinline__ void mate_values(const uint4& v, const uint64_t (&own)[4], int mate, uint64_t (&m)[4]) {
    if constexpr (INTER) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo, hi;
            f2_unpack(own[k], lo, hi);
            m[k] = f2_pack(hi, lo);
        }
    } else {
        unpack8(shfl4(v, mate), m);
    }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kNrThreads, 3) norm_rope_kernel(const NormRopeParams p) {
    constexpr int LPR = D / 8;
    constexpr int G = kNrThreads / LPR;  // lane groups of the block
    constexpr int U = 4;                 // rows in flight per group
    const LaneMap<D> lm(p.R, INTER);
    const int group = threadIdx.x / LPR;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tb;
    const int tt = group % p.tb, off = group / p.tb, hstep = G / p.tb;
    const bool live = tok0 + tt < p.ntokens;
    const int64_t tok = live ? tok0 + tt : 0;
    const int h0 = static_cast<int>(blockIdx.y) * p.hb, h1 = min(h0 + p.hb, p.Hq + p.Hkv);
    const int64_t b = tok / p.T, t = tok % p.T;
    const __nv_bfloat16* src = nullptr;   // this lane's dims of its next row to load
    __nv_bfloat16* dst = nullptr;         // and of its next row to store
    int64_t sstep = 0, dstep = 0;
    int n = 0, todo = 0;                  // rows of the section that are left to load, and its rounds
    uint4 v[U];
    // heads [lo, hi) of one side: the first U rows travel
    auto begin = [&](bool is_k) {
        const int lo = is_k ? max(h0 - p.Hq, 0) : h0, hi = is_k ? h1 - p.Hq : min(h1, p.Hq);
        const int64_t* st = is_k ? p.xk : p.xq;
        const int64_t H = is_k ? p.Hkv : p.Hq;
        src = (is_k ? p.Xk : p.Xq) + b * st[0] + t * st[1] + (lo + off) * st[2] + 8 * lm.lane8;
        dst = (is_k ? p.K : p.Q) + ((b * H + lo + off) * p.T + t) * D + 8 * lm.lane8;
        sstep = hstep * st[2];
        dstep = static_cast<int64_t>(hstep) * p.T * D;
        n = live ? (hi - lo - off + hstep - 1) / hstep : 0;
        todo = hi > lo ? (hi - lo + hstep - 1) / hstep : 0;  // the same for every group of the block
        if (hi - lo - off <= 0) n = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u < n) v[u] = load_row(src);
            src += sstep;
        }
    };
    const bool has_q = h0 < p.Hq;
    begin(!has_q);  // before the angles are formed
    Turn tn;
    form_turn<D, INTER>(p, lm, tok, tn);
    for (int side = has_q ? 0 : 1; side < 2; ++side) {
        if (side == 1 && has_q) {
            if (h1 <= p.Hq) break;
            begin(true);
        }
        // y = r (x a + x_mate c)
        const float* w = side == 0 ? p.wq : p.wk;
        const int md = INTER ? 0 : (lm.mate - static_cast<int>(threadIdx.x & 31)) * 8;
        uint64_t a[4], c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float wa[2] = {1.f, 1.f}, wm[2] = {1.f, 1.f};
            if (w != nullptr) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = 8 * lm.lane8 + 2 * k + e;
                    wa[e] = __ldg(w + d);
                    wm[e] = __ldg(w + (INTER ? d ^ 1 : d + md));
                }
            }
            a[k] = f2_pack(tn.c[2 * k] * wa[0], tn.c[2 * k + 1] * wa[1]);
            c[k] = f2_pack(tn.s[2 * k] * wm[0], tn.s[2 * k + 1] * wm[1]);
        }
        // every lane of a warp walks the same number of rows: the shuffles need all of them
        for (int i = 0; i < todo; i += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u >= todo) break;
                const bool ok = i + u < n;
                if (!ok) v[u] = make_uint4(0u, 0u, 0u, 0u);
                uint64_t x[4], m[4];
                unpack8(v[u], x);
                mate_values<INTER>(v[u], x, lm.mate, m);
                uint64_t s2 = f2_mul(x[0], x[0]);
#pragma unroll
                for (int k = 1; k < 4; ++k) s2 = nr_fma2(x[k], x[k], s2);
                float s0, s1;
                f2_unpack(s2, s0, s1);
                const float r = rsqrtf(row_sum<D>(s0 + s1) * (1.f / D) + p.eps);
                const uint64_t r2 = f2_pack(r, r);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = f2_mul(nr_fma2(m[k], c[k], f2_mul(x[k], a[k])), r2);
                if (ok) *reinterpret_cast<uint4*>(dst) = pack8(x);
                dst += dstep;
                if (i + u + U < n) v[u] = load_row(src);
                src += sstep;
            }
        }
    }
}

// One side (queries or keys) per block: blocks [0, p.qblocks) walk the query tiles, the others the
// key tiles, so a thread has one side's weights and sums.
template <int D, bool INTER>
__global__ void __launch_bounds__(kNrThreads, 2) norm_rope_backward_kernel(const NormRopeParams p) {
    __shared__ float red[kNrThreads * 8];
    constexpr int LPR = D / 8;
    constexpr int G = kNrThreads / LPR;
    constexpr int U = 4;
    const LaneMap<D> lm(p.R, INTER);
    const int group = threadIdx.x / LPR;
    const int tt = group % p.tb, off = group / p.tb, hstep = G / p.tb;
    const bool is_k = static_cast<int>(blockIdx.x) >= p.qblocks;
    const int H = is_k ? p.Hkv : p.Hq;
    const int hb = is_k ? p.hbk : p.hb, hsplits = (H + hb - 1) / hb;
    const int64_t tiles = (p.ntokens + p.tb - 1) / p.tb * hsplits;
    const int64_t* st = is_k ? p.xk : p.xq;
    const int64_t* gt = is_k ? p.dxk : p.dxq;
    const float* w = is_k ? p.wk : p.wq;
    uint64_t wl[4], g2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int d = 8 * lm.lane8 + 2 * k;
        wl[k] = w != nullptr ? f2_pack(__ldg(w + d), __ldg(w + d + 1)) : f2_pack(1.f, 1.f);
        g2[k] = 0ull;
    }
    const int first = static_cast<int>(blockIdx.x) - (is_k ? p.qblocks : 0);
    const int step = is_k ? static_cast<int>(gridDim.x) - p.qblocks : p.qblocks;
    for (int64_t tile = first; tile < tiles; tile += step) {
        const int64_t tok0 = (tile / hsplits) * p.tb;
        const bool live = tok0 + tt < p.ntokens;
        const int64_t tok = live ? tok0 + tt : 0;
        const int h0 = static_cast<int>(tile % hsplits) * hb, h1 = min(h0 + hb, H);
        const int64_t b = tok / p.T, t = tok % p.T;
        const __nv_bfloat16* xs = (is_k ? p.Xk : p.Xq) + b * st[0] + t * st[1] + (h0 + off) * st[2] + 8 * lm.lane8;
        const __nv_bfloat16* gs = (is_k ? p.dK : p.dQ) + ((b * H + h0 + off) * p.T + t) * D + 8 * lm.lane8;
        __nv_bfloat16* dst = (is_k ? p.dXk : p.dXq) + b * gt[0] + t * gt[1] + (h0 + off) * gt[2] + 8 * lm.lane8;
        const int64_t sstep = hstep * st[2], gstep = static_cast<int64_t>(hstep) * p.T * D, dstep = hstep * gt[2];
        const int n = live && h1 - h0 > off ? (h1 - h0 - off + hstep - 1) / hstep : 0;
        const int todo = (h1 - h0 + hstep - 1) / hstep;
        uint4 xv[U], gv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u < n) {
                xv[u] = load_row(xs);
                gv[u] = load_row(gs);
            }
            xs += sstep;
            gs += gstep;
        }
        Turn tn;
        form_turn<D, INTER>(p, lm, tok, tn);
        for (int i = 0; i < todo; i += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u >= todo) break;
                const bool ok = i + u < n;
                if (!ok) xv[u] = gv[u] = make_uint4(0u, 0u, 0u, 0u);
                uint64_t x[4], g[4], m[4];
                unpack8(xv[u], x);
                unpack8(gv[u], g);
                mate_values<INTER>(gv[u], g, lm.mate, m);
                uint64_t s2 = 0ull, d2 = 0ull;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // du: the turn taken back; then dn = du w
                    g[k] = nr_fma2(m[k], f2_pack(-tn.s[2 * k], -tn.s[2 * k + 1]),
                                   f2_mul(g[k], f2_pack(tn.c[2 * k], tn.c[2 * k + 1])));
                    m[k] = f2_mul(g[k], wl[k]);
                    s2 = nr_fma2(x[k], x[k], s2);
                    d2 = nr_fma2(m[k], x[k], d2);
                }
                float s0, s1, d0, d1;
                f2_unpack(s2, s0, s1);
                f2_unpack(d2, d0, d1);
                const float ss = row_sum<D>(s0 + s1), dot = row_sum<D>(d0 + d1);
                // a row that does not count adds nothing (with eps = 0 its own r would be infinite)
                const float r = ok ? rsqrtf(ss * (1.f / D) + p.eps) : 0.f;
                const float f = -r * r * dot * (1.f / D);
                const uint64_t r2 = f2_pack(r, r), f2 = f2_pack(f, f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    m[k] = f2_mul(nr_fma2(x[k], f2, m[k]), r2);
                    g2[k] = nr_fma2(g[k], f2_mul(x[k], r2), g2[k]);
                }
                if (ok) *reinterpret_cast<uint4*>(dst) = pack8(m);
                dst += dstep;
                if (i + u + U < n) {
                    xv[u] = load_row(xs);
                    gv[u] = load_row(gs);
                }
                xs += sstep;
                gs += gstep;
            }
        }
    }
    // the block's groups: one row of partial sums per block
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        f2_unpack(g2[k], lo, hi);
        red[group * D + 8 * lm.lane8 + 2 * k] = lo;
        red[group * D + 8 * lm.lane8 + 2 * k + 1] = hi;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kNrThreads) {
        float s = 0.f;
#pragma unroll 4
        for (int gg = 0; gg < G; ++gg) s += red[gg * D + d];
        p.part[static_cast<int64_t>(blockIdx.x) * D + d] = s;
    }
}

// dwq and dwk from the blocks' partial sums [blocks][D]: 32 columns per block (blockIdx.y: the side),
// 32 threads per column.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int qblocks, int blocks, int D, float* dwq,
                                                            float* dwk) {
    __shared__ float red[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), ty = threadIdx.x >> 5;
    const int lo = blockIdx.y == 0 ? 0 : qblocks, hi = blockIdx.y == 0 ? qblocks : blocks;
    float s = 0.f;
#pragma unroll 8
    for (int i = lo + ty; i < hi; i += 32) s += __ldcg(part + static_cast<int64_t>(i) * D + col);
    red[ty][threadIdx.x & 31] = s;
    __syncthreads();
    if (ty == 0) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += red[i][threadIdx.x];
        float* dst = blockIdx.y == 0 ? dwq : dwk;
        if (dst != nullptr) dst[col] = v;
    }
}

// Tokens per tile and heads per tile: full tiles (one token per lane group, all heads) unless that
// gives fewer than two blocks per SM; then fewer tokens, then fewer heads, down to one row per lane
// group.
static int64_t norm_rope_tiles(NormRopeParams* p, int D, int H) {
    const int G = kNrThreads / (D / 8);
    p->tb = G;
    p->hb = H;
    while (true) {
        const int64_t blocks = (p->ntokens + p->tb - 1) / p->tb * ((H + p->hb - 1) / p->hb);
        if (blocks >= kNormRopeBlocks / 2) return blocks;
        if (p->tb > 1)
            p->tb /= 2;
        else if (p->hb > G)
            p->hb = (p->hb + 1) / 2;
        else
            return blocks;
    }
}

bool launch_norm_rope(NormRopeParams p, int D, bool inter, cudaStream_t st) {
    norm_rope_tiles(&p, D, p.Hq + p.Hkv);
    const int64_t bx = (p.ntokens + p.tb - 1) / p.tb;
    if (bx > INT32_MAX) return false;
    const dim3 grid(static_cast<unsigned>(bx), (p.Hq + p.Hkv + p.hb - 1) / p.hb);
    if (D == 64) {
        if (inter)
            norm_rope_kernel<64, true><<<grid, kNrThreads, 0, st>>>(p);
        else
            norm_rope_kernel<64, false><<<grid, kNrThreads, 0, st>>>(p);
    } else {
        if (inter)
            norm_rope_kernel<128, true><<<grid, kNrThreads, 0, st>>>(p);
        else
            norm_rope_kernel<128, false><<<grid, kNrThreads, 0, st>>>(p);
    }
    return cudaGetLastError() == cudaSuccess;
}

bool launch_norm_rope_backward(NormRopeParams p, int D, bool inter, float* dwq, float* dwk, cudaStream_t st,
                               int32_t* launches) {
    // the tile shape of all heads together; the blocks are shared out by the sides' rows
    const int H = p.Hq + p.Hkv;
    const int64_t all = norm_rope_tiles(&p, D, H);
    p.hbk = p.hb < p.Hkv ? p.hb : p.Hkv;
    p.hb = p.hb < p.Hq ? p.hb : p.Hq;
    const int64_t tt = (p.ntokens + p.tb - 1) / p.tb;
    const int64_t qtiles = tt * ((p.Hq + p.hb - 1) / p.hb), ktiles = tt * ((p.Hkv + p.hbk - 1) / p.hbk);
    const int64_t most = all < kNormRopeBlocks ? all + 1 : kNormRopeBlocks;
    int64_t qb = (most * p.Hq + H - 1) / H;
    if (qb >= most) qb = most - 1;
    if (qb < 1) qb = 1;
    int64_t kb = most - qb < 1 ? 1 : most - qb;
    if (qb > qtiles) qb = qtiles;
    if (kb > ktiles) kb = ktiles;
    p.qblocks = static_cast<int>(qb);
    const int grid = static_cast<int>(qb + kb);
    if (D == 64) {
        if (inter)
            norm_rope_backward_kernel<64, true><<<grid, kNrThreads, 0, st>>>(p);
        else
            norm_rope_backward_kernel<64, false><<<grid, kNrThreads, 0, st>>>(p);
    } else {
        if (inter)
            norm_rope_backward_kernel<128, true><<<grid, kNrThreads, 0, st>>>(p);
        else
            norm_rope_backward_kernel<128, false><<<grid, kNrThreads, 0, st>>>(p);
    }
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    if (dwq == nullptr && dwk == nullptr) return true;
    // The rows' kernel does not trigger it early, so it starts when the last block has exited; what the attribute saves is
    // the launch itself. It waits for the rows' sums all the same.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(D / 32), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(p.part), p.qblocks, grid, D, dwq, dwk) !=
        cudaSuccess)
        return false;
    ++*launches;
    return true;
}

}  // namespace pisa
