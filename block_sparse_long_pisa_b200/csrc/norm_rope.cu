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
//     are formed once per block and not once per head. The angle is pos * inv_freq in fp64, taken
//     modulo one turn before it is rounded to fp32: a far position keeps its phase (an fp32 product
//     is off by 2^-24 of an angle of 10^6, 0.06 rad).
//   * A tile is as many tokens as a block has lane groups: the tile's stores of one head are one
//     contiguous run (16 rows of 256 bytes at D = 128) although input and output orders differ.
//   * Few tokens (one decode step): tiles shrink to one token and its heads split over blocks, down
//     to one row per lane group, until the grid fills the SMs.
// The weight gradients are summed in registers along a block's tiles (a grid of at most
// kNormRopeBlocks blocks), then over the block's groups through shared memory, then over the blocks
// by a second kernel: fixed orders, no atomics.
#include <cuda_bf16.h>

#include "pisa_device.cuh"

namespace pisa {

constexpr int kNrThreads = 256;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = bf_lo(w[k]);
        f[2 * k + 1] = bf_hi(w[k]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
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

template <int D>
__device__ __forceinline__ void load_turn(const float2* tab, const LaneMap<D>& lm, int R, bool inter, Turn& t) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        t.c[k] = 1.f;
        t.s[k] = 0.f;
    }
    if (!lm.turns) return;
    if (inter) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 cs = tab[4 * lm.lane8 + k];
            t.c[2 * k] = t.c[2 * k + 1] = cs.x;
            t.s[2 * k] = -cs.y;
            t.s[2 * k + 1] = cs.y;
        }
    } else {
        const int i0 = 8 * lm.lane8 - (lm.second ? R / 2 : 0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 cs = tab[i0 + k];
            t.c[k] = cs.x;
            t.s[k] = lm.second ? cs.y : -cs.y;
        }
    }
}

// The mates' values of this lane's 8 dims.
__device__ __forceinline__ void mate_values(const uint4& v, int mate, bool inter, float (&m)[8]) {
    if (inter) {
        unpack8(make_uint4(__funnelshift_l(v.x, v.x, 16), __funnelshift_l(v.y, v.y, 16),
                           __funnelshift_l(v.z, v.z, 16), __funnelshift_l(v.w, v.w, 16)), m);
    } else {
        unpack8(shfl4(v, mate), m);
    }
}

// cos and sin of the tile's tokens: tab[token in tile][i], i < R/2.
__device__ __forceinline__ void fill_table(const NormRopeParams& p, int64_t tok0, int ntok, float2* tab) {
    const int half = p.R / 2;
    for (int e = threadIdx.x; e < ntok * half; e += kNrThreads) {
        const int tt = e / half, i = e % half;
        if (tok0 + tt >= p.ntokens) break;
        const double turns = static_cast<double>(p.pos[tok0 + tt]) * static_cast<double>(p.inv_freq[i]) *
                             0.15915494309189533577;
        const float frac = static_cast<float>(turns - rint(turns));
        float s, c;
        sincospif(2.f * frac, &s, &c);
        tab[tt * half + i] = make_float2(c, s);
    }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
    extern __shared__ __align__(16) float2 tab[];
    constexpr int LPR = D / 8;
    constexpr int G = kNrThreads / LPR;  // lane groups of the block
    constexpr int U = 4;                 // rows in flight per group
    const LaneMap<D> lm(p.R, INTER);
    const int group = threadIdx.x / LPR;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tb;
    const int tt = group % p.tb;
    const int64_t tok = tok0 + tt;
    const bool live = tok < p.ntokens;
    const int hstep = G / p.tb;
    const int h0 = static_cast<int>(blockIdx.y) * p.hb, h1 = min(h0 + p.hb, p.Hq + p.Hkv);
    const int64_t b = live ? tok / p.T : 0, t = live ? tok % p.T : 0;
    const int64_t xq0 = b * p.xq[0] + t * p.xq[1] + 8 * lm.lane8, xk0 = b * p.xk[0] + t * p.xk[1] + 8 * lm.lane8;
    auto src = [&](int h) -> const __nv_bfloat16* {
        return h < p.Hq ? p.Xq + xq0 + h * p.xq[2] : p.Xk + xk0 + (h - p.Hq) * p.xk[2];
    };
    const int hfirst = h0 + group / p.tb;
    // the first rows travel while the angles are formed
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (live && hfirst + u * hstep < h1) v[u] = load_row(src(hfirst + u * hstep));
    fill_table(p, tok0, p.tb, tab);
    __syncthreads();
    Turn tn;
    load_turn<D>(tab + (live ? tt : 0) * (p.R / 2), lm, p.R, INTER, tn);

    float a[8], bb[8];
    bool for_k = false;
    auto fold = [&](const float* w) {
        const int md = INTER ? 0 : (lm.mate - static_cast<int>(threadIdx.x & 31)) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int d = 8 * lm.lane8 + k;
            const int m = INTER ? (lm.turns ? (d ^ 1) : d) : d + md;
            a[k] = tn.c[k] * (w != nullptr ? __ldg(w + d) : 1.f);
            bb[k] = tn.s[k] * (w != nullptr ? __ldg(w + m) : 1.f);
        }
    };
    fold(p.wq);
    // every lane of a warp walks the same number of rows: the shuffles need all of them
    for (int h = h0; h < h1; h += U * hstep) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hh = h + u * hstep + group / p.tb;
            const bool ok = live && hh < h1;
            if (ok && hh >= p.Hq && !for_k) {
                fold(p.wk);
                for_k = true;
            }
            if (!ok) v[u] = make_uint4(0u, 0u, 0u, 0u);
            float x[8], m[8], y[8];
            unpack8(v[u], x);
            mate_values(v[u], lm.mate, INTER, m);
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
            const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + p.eps);
            // past the rotated dims b is 0: the mate (the lane itself) must not bring in a NaN twice,
            // which is harmless, its own value being one already
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = r * fmaf(m[k], bb[k], x[k] * a[k]);
            if (ok) {
                __nv_bfloat16* dst = hh < p.Hq ? p.Q + ((b * p.Hq + hh) * p.T + t) * D
                                               : p.K + ((b * p.Hkv + (hh - p.Hq)) * p.T + t) * D;
                *reinterpret_cast<uint4*>(dst + 8 * lm.lane8) = pack8(y);
            }
            const int hn = hh + U * hstep;
            if (live && hn < h1) v[u] = load_row(src(hn));
        }
    }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kNrThreads) norm_rope_backward_kernel(const NormRopeParams p) {
    extern __shared__ __align__(16) float2 tab[];
    __shared__ float red[kNrThreads * 8];
    constexpr int LPR = D / 8;
    constexpr int G = kNrThreads / LPR;
    constexpr int U = 2;
    const LaneMap<D> lm(p.R, INTER);
    const int group = threadIdx.x / LPR;
    const int tt = group % p.tb;
    const int hstep = G / p.tb;
    const int hsplits = (p.Hq + p.Hkv + p.hb - 1) / p.hb;
    float wq[8], wk[8], gq[8], gk[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        wq[k] = p.wq != nullptr ? __ldg(p.wq + 8 * lm.lane8 + k) : 1.f;
        wk[k] = p.wk != nullptr ? __ldg(p.wk + 8 * lm.lane8 + k) : 1.f;
        gq[k] = gk[k] = 0.f;
    }
    for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const int64_t tok0 = (tile / hsplits) * p.tb;
        const int64_t tok = tok0 + tt;
        const bool live = tok < p.ntokens;
        const int h0 = static_cast<int>(tile % hsplits) * p.hb, h1 = min(h0 + p.hb, p.Hq + p.Hkv);
        const int64_t b = live ? tok / p.T : 0, t = live ? tok % p.T : 0;
        const int64_t c0 = 8 * lm.lane8;
        auto load = [&](int h, uint4& x, uint4& g) {
            if (h < p.Hq) {
                x = load_row(p.Xq + b * p.xq[0] + t * p.xq[1] + h * p.xq[2] + c0);
                g = load_row(p.dQ + ((b * p.Hq + h) * p.T + t) * D + c0);
            } else {
                const int hk = h - p.Hq;
                x = load_row(p.Xk + b * p.xk[0] + t * p.xk[1] + hk * p.xk[2] + c0);
                g = load_row(p.dK + ((b * p.Hkv + hk) * p.T + t) * D + c0);
            }
        };
        uint4 xv[U], gv[U];
        const int hfirst = h0 + group / p.tb;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (live && hfirst + u * hstep < h1) load(hfirst + u * hstep, xv[u], gv[u]);
        __syncthreads();  // the previous tile's table has been read
        fill_table(p, tok0, p.tb, tab);
        __syncthreads();
        Turn tn;
        load_turn<D>(tab + (live ? tt : 0) * (p.R / 2), lm, p.R, INTER, tn);
        for (int h = h0; h < h1; h += U * hstep) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hh = h + u * hstep + group / p.tb;
                const bool ok = live && hh < h1;
                const bool is_q = hh < p.Hq;
                if (!ok) xv[u] = gv[u] = make_uint4(0u, 0u, 0u, 0u);
                float x[8], g[8], m[8], dn[8];
                unpack8(xv[u], x);
                unpack8(gv[u], g);
                mate_values(gv[u], lm.mate, INTER, m);
                float ss = 0.f, dot = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    g[k] = fmaf(m[k], -tn.s[k], g[k] * tn.c[k]);  // du: the turn taken back
                    dn[k] = g[k] * (is_q ? wq[k] : wk[k]);
                    ss = fmaf(x[k], x[k], ss);
                    dot = fmaf(dn[k], x[k], dot);
                }
                ss = row_sum<D>(ss);
                dot = row_sum<D>(dot);
                const float r = rsqrtf(ss * (1.f / D) + p.eps);
                const float f = r * r * dot * (1.f / D);
                if (ok) {
                    float dx[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        dx[k] = r * fmaf(-f, x[k], dn[k]);
                        const float xr = x[k] * r;
                        if (is_q)
                            gq[k] = fmaf(g[k], xr, gq[k]);
                        else
                            gk[k] = fmaf(g[k], xr, gk[k]);
                    }
                    __nv_bfloat16* dst = is_q ? p.dXq + b * p.dxq[0] + t * p.dxq[1] + hh * p.dxq[2]
                                              : p.dXk + b * p.dxk[0] + t * p.dxk[1] + (hh - p.Hq) * p.dxk[2];
                    *reinterpret_cast<uint4*>(dst + c0) = pack8(dx);
                }
                const int hn = hh + U * hstep;
                if (live && hn < h1) load(hn, xv[u], gv[u]);
            }
        }
    }
    // the block's groups, then one row of partial sums per block: [block][q, k][D]
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) red[group * D + 8 * lm.lane8 + k] = side == 0 ? gq[k] : gk[k];
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += kNrThreads) {
            float s = 0.f;
#pragma unroll 4
            for (int gg = 0; gg < G; ++gg) s += red[gg * D + d];
            p.part[(static_cast<int64_t>(blockIdx.x) * 2 + side) * D + d] = s;
        }
    }
}

// dwq and dwk from the blocks' partial sums: 32 columns per block, 32 threads per column.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int blocks, int D, float* dwq,
                                                            float* dwk) {
    __shared__ float red[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), ty = threadIdx.x >> 5;
    float s = 0.f;
    for (int i = ty; i < blocks; i += 32) s += part[static_cast<int64_t>(i) * 2 * D + col];
    red[ty][threadIdx.x & 31] = s;
    __syncthreads();
    if (ty == 0) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += red[i][threadIdx.x];
        float* dst = col < D ? dwq : dwk;
        if (dst != nullptr) dst[col % D] = v;
    }
}

// Tokens per tile and heads per tile: full tiles (one token per lane group, all heads) unless that
// leaves SMs idle; then fewer tokens, then fewer heads, down to one row per lane group.
void norm_rope_tiles(NormRopeParams* p, int D) {
    const int G = kNrThreads / (D / 8), H = p->Hq + p->Hkv;
    p->tb = G;
    p->hb = H;
    while (true) {
        const int64_t blocks = (p->ntokens + p->tb - 1) / p->tb * ((H + p->hb - 1) / p->hb);
        if (blocks >= kNormRopeBlocks) break;
        if (p->tb > 1)
            p->tb /= 2;
        else if (p->hb > G)
            p->hb = (p->hb + 1) / 2;
        else
            break;
    }
    p->tiles = (p->ntokens + p->tb - 1) / p->tb * ((H + p->hb - 1) / p->hb);
}

bool launch_norm_rope(NormRopeParams p, int D, bool inter, cudaStream_t st) {
    norm_rope_tiles(&p, D);
    const int64_t bx = (p.ntokens + p.tb - 1) / p.tb;
    if (bx > INT32_MAX) return false;
    const dim3 grid(static_cast<unsigned>(bx), (p.Hq + p.Hkv + p.hb - 1) / p.hb);
    const size_t smem = static_cast<size_t>(p.tb) * (p.R / 2) * sizeof(float2);
    if (D == 64) {
        if (inter)
            norm_rope_kernel<64, true><<<grid, kNrThreads, smem, st>>>(p);
        else
            norm_rope_kernel<64, false><<<grid, kNrThreads, smem, st>>>(p);
    } else {
        if (inter)
            norm_rope_kernel<128, true><<<grid, kNrThreads, smem, st>>>(p);
        else
            norm_rope_kernel<128, false><<<grid, kNrThreads, smem, st>>>(p);
    }
    return cudaGetLastError() == cudaSuccess;
}

bool launch_norm_rope_backward(NormRopeParams p, int D, bool inter, float* dwq, float* dwk, cudaStream_t st,
                               int32_t* launches) {
    norm_rope_tiles(&p, D);
    const int grid = static_cast<int>(p.tiles < kNormRopeBlocks ? p.tiles : kNormRopeBlocks);
    const size_t smem = static_cast<size_t>(p.tb) * (p.R / 2) * sizeof(float2);
    if (D == 64) {
        if (inter)
            norm_rope_backward_kernel<64, true><<<grid, kNrThreads, smem, st>>>(p);
        else
            norm_rope_backward_kernel<64, false><<<grid, kNrThreads, smem, st>>>(p);
    } else {
        if (inter)
            norm_rope_backward_kernel<128, true><<<grid, kNrThreads, smem, st>>>(p);
        else
            norm_rope_backward_kernel<128, false><<<grid, kNrThreads, smem, st>>>(p);
    }
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    if (dwq == nullptr && dwk == nullptr) return true;
    norm_rope_dw_kernel<<<2 * D / 32, 1024, 0, st>>>(p.part, grid, D, dwq, dwk);
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    return true;
}

}  // namespace pisa
