// Attention of a tree of drafted tokens over a K/V cache (one drafted token is plain decode).
//
//   rows   the T drafted tokens of the gh query heads that share a selection row: gh * T rows
//   keys   the cache in units of 64 keys (selected blocks and tail, or all of it, up to the sequence's
//          length), and last the drafted tokens themselves, masked by their ancestor bits
//   O = softmax(scale Q K^T) V with a running maximum and sum (fp32); no score leaves the SM
//
// Two kernels share the work by the rows that a key serves: up to 16, where the bytes of the cache are
// all that should count (attn_tree_few.cu, mma.sync), and more, where the products and exponentials count
// too (attn_tree_many.cu, tcgen05).
//
// Work split (pisa_tree.cuh). Sequences have unlike lengths that only the device knows, so the units of
// all row tiles are laid end to end and cut into equal runs, one per CTA of a fixed grid; a run may end
// one row tile, hold whole ones and begin another. A row tile inside one run is finished there; one that
// crosses runs leaves partial (o, m, l) that attn_tree_merge_kernel joins in run order. Every CTA finds
// its run by summing the lengths itself: no scheduling pass, no atomics in any sum, and the same inputs
// give the same bits.
//
// This file: the join, and the choice of the kernel.
#include <cuda_bf16.h>

#include "pisa_device.cuh"
#include "pisa_tree.cuh"

namespace pisa {

constexpr unsigned kMergeBlocks = 148 * 12;

// Joins the pieces of the row tiles that crossed runs, in run order: m = max m_i, weights
// 2^(m_i - m). grid: (row tiles, shares of their rows); 128 threads, one float4 of a row each (D = 128), a warp a
// row at a time. Bound by latency and, before the wait, by the 64-bit divisions that find the runs: those are paid
// once a warp, not once a row (64 tokens of four heads in 512 row tiles, the runs included: 396 us, 473 us with a
// warp for every row).
template <int D>
__global__ void __launch_bounds__(128) attn_tree_merge_kernel(const TreeParams p, int RM) {
    const int64_t tile = blockIdx.x;
    const int b = static_cast<int>(tile / p.rows_per_seq);
    const int rem = static_cast<int>(tile % p.rows_per_seq);
    const int hs = rem / p.mt, row_base = (rem % p.mt) * p.rpt;
    const int rows = min(p.rpt, p.gh * p.T - row_base);
    // (what comes before the wait reads the lengths alone, which were there before the runs began)
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
    // the pieces: 2 c0 + 1, then 2 (c0 + 1), 2 (c0 + 2), ..
    const int stride = RM * (D + 2), pieces = static_cast<int>(c1 - c0) + 1;
    const float* part = p.part + (2 * c0 + 1) * stride;
    auto slot = [&](int i) { return part + static_cast<int64_t>(max(2 * i - 1, 0)) * stride; };
    const int64_t orow0 = (static_cast<int64_t>(b) * p.Hq + hs * p.gh) * p.T + row_base;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // also by a block without rows: the grid ends after the runs
    if (pieces == 1) return;
#pragma unroll 1
    for (int row = static_cast<int>(blockIdx.y * 4 + (threadIdx.x >> 5)); row < rows; row += static_cast<int>(gridDim.y * 4)) {
        // (m, l) of piece i in lane i % 32
        auto ml_of = [&](int i) {
            return i < pieces ? *reinterpret_cast<const float2*>(slot(i) + RM * D + 2 * row) : make_float2(-INFINITY, 0.f);
        };
        const float2 ml0 = ml_of(lane);
        float M = ml0.x;
        for (int i = 32 + lane; i < pieces; i += 32) M = fmaxf(M, ml_of(i).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
        constexpr int V = D / 32;  // values of the row per lane
        float acc[V], l = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        for (int i0 = 0; i0 < pieces; i0 += 32) {
            const float2 ml = i0 == 0 ? ml0 : ml_of(i0 + lane);
            const float mine = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : fast_exp2(ml.x - M);
#pragma unroll 8
            for (int i = i0; i < min(pieces, i0 + 32); ++i) {
                const float* s = slot(i) + row * D;
                float v[V];
                if constexpr (V == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(s + 4 * lane);
                    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(s + 2 * lane);
                    v[0] = x.x, v[1] = x.y;
                }
                const float w = __shfl_sync(0xFFFFFFFFu, mine, i - i0);
                l += w * __shfl_sync(0xFFFFFFFFu, ml.y, i - i0);
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += w * v[k];
            }
        }
        const int64_t orow = orow0 + row;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if constexpr (V == 4)
            *reinterpret_cast<uint2*>(p.O + orow * D + 4 * lane) =
                make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<uint32_t*>(p.O + orow * D + 2 * lane) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
        if (lane == 0 && p.lse != nullptr)
            p.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
    }
}

// ---------------------------------------------------------------- host side

// Rows of one row tile for a selection row of `rows` rows, T drafted tokens: 8 or 16 (attn_tree_few.cu), 128 or
// 256 (attn_tree_many.cu); where a tile does not hold them several share them evenly. Up to 32 rows over an
// e4m3 cache are two tiles of 16 (each reads the cache): 64 caches of 8 heads, 64 blocks of 64 keys selected, eight
// tokens of four heads, 276 us against 317 us as one tile of 128. A third tile would lose (nine tokens, 399 us
// against 320 us), and so would two over a bf16 cache (351 us against 221 us).
int tree_row_tile(int rows, int T, bool e4m3) {
    if (rows <= 8) return 8;
    if (rows <= 16 || (e4m3 && rows <= 32 && T <= 16)) return 16;
    return rows <= 128 ? 128 : 256;
}

// CTAs on one SM: as many as its shared memory takes.
int tree_ctas_per_sm(int rm, bool e4m3) { return rm > 16 ? 1 : e4m3 && rm == 8 ? 3 : 2; }

bool launch_tree_merge(const TreeParams& p, int D, int rm, cudaStream_t st, int32_t* launches) {
    cudaLaunchConfig_t cfg{};
    // blocks enough to fill the SMs, and no more than rows
    const unsigned tiles = static_cast<unsigned>(p.B) * p.rows_per_seq, shares = (p.rpt + 3) / 4;
    const unsigned want = tiles < kMergeBlocks ? (kMergeBlocks + tiles - 1) / tiles : 1;
    cfg.gridDim = dim3(tiles, want < shares ? want : shares);
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

bool launch_attn_tree(const TreeParams& p, int D, bool e4m3, int rm, const void* K, const void* Kc, const void* Vc,
                      cudaStream_t st, int32_t* launches) {
    return rm <= 16 ? launch_attn_tree_few(p, D, e4m3, rm, K, Kc, Vc, st, launches)
                    : launch_attn_tree_many(p, D, e4m3, rm, K, Kc, Vc, st, launches);
}

}  // namespace pisa
