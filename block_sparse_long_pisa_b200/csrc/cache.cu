// K/V cache rows: quantised as they are written, read back, and pooled into the key pyramid.
//
// A row of an e4m3 cache is D bytes and one exponent byte e; its values are byte values times
// 2^(e - 127). The scale is a power of two, so scaling is exact and each value is rounded once; a
// scale max|x| / 448 would round twice and gain nothing, the format's relative step being the same
// in every binade. One byte per row (not four) is 0.8 % of a 128-value row.
//
// All three kernels are bound by HBM (write: 2 bytes read and 1 written per value; read: the other
// way round; pooling: 1 byte read). D/8 lanes hold a row, 8 values each: one 16-byte bf16 access
// and one 8-byte e4m3 access per lane, and the row's largest magnitude is a maximum over integer
// words (bf16 magnitudes order like their bits) and log2(D/8) shuffles. Each lane group keeps
// several rows in flight.
//
// Measured (8 heads of 128, e4m3): write of 131,072 tokens 0.81 GB in 120 us, 6.7 TB/s, the copy rate (two rows
// share a word in the maximum's shuffles and pairs are scaled at once: 158 us with a word a row, at 67 % of the
// issue slots); write of one token to each of 64 sequences 2.2 us; read of 7 ragged prefixes 0.29 GB in 48 us,
// 6.0 TB/s (91 %); pyramids of 8 caches of 32,768 keys 0.29 GB in 60 us, 4.9 TB/s (75 %; issue 58 %: two
// conversions and a fused multiplication for two values that are two bytes).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pisa_device.cuh"
#include "pisa_pool.cuh"

namespace pisa {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 4;  // rows of one lane group, all in flight together

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The two e4m3 values of a word's low (HI: high) half.
template <bool HI>
__device__ __forceinline__ float2 e4m3x2_values(uint32_t word) {
    const uint32_t h = e4m3x2_f16x2<HI>(word);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 2^(e - 127) of an exponent byte 1 .. 254; 255 gives an infinity, which times a zero byte is the
// NaN that such a row stands for.
__device__ __forceinline__ float exp_value(uint32_t e) { return __uint_as_float(e << 23); }

// A lane group's segment: kCacheRows consecutive tokens of one plane, clipped to the tokens that count;
// segments of a plane lie side by side. One division and one look at start and count per segment.
struct Segment {
    int b, h, t0, n;       // sequence, head, first token, tokens that count (0: nothing to do)
    int64_t at;            // cache row of the first token
    __device__ __forceinline__ Segment(const CacheParams& p, uint32_t seg, uint32_t detail, bool reports) {
        const uint32_t per_plane = (static_cast<uint32_t>(p.tokens) + kCacheRows - 1) / kCacheRows;
        const uint32_t plane = seg / per_plane;
        b = h = t0 = n = 0;
        at = 0;
        if (plane >= static_cast<uint32_t>(p.B) * p.H) return;
        b = static_cast<int>(plane / static_cast<uint32_t>(p.H));
        h = static_cast<int>(plane - static_cast<uint32_t>(b) * p.H);
        t0 = static_cast<int>(seg - plane * per_plane) * kCacheRows;
        const int64_t start = p.start != nullptr ? __ldg(p.start + b) : 0;
        const int count = p.count != nullptr ? __ldg(p.count + b) : p.tokens;
        if (count < 0 || count > p.tokens || start < 0 || start + count > p.cap) {
            // the sequence is left alone
            if (reports && h == 0 && t0 == 0) record_error(p.status, PISA_ERR_BAD_INDEX, detail);
            return;
        }
        n = max(0, min(kCacheRows, count - t0));
        at = static_cast<int64_t>(plane) * p.cap + start + t0;
    }
};

// grid: (segment blocks, K or V).
template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
    constexpr int LPR = D / 8, G = kCacheThreads / LPR;
    const int lane8 = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const bool is_v = blockIdx.y != 0;
    const Segment w(p, blockIdx.x * G + group, (kKernCache << 8) | 0xB0u, lane8 == 0 && !is_v);
    const int64_t* st = is_v ? p.vs : p.ks;
    const int64_t step = st[2];
    const __nv_bfloat16* src = (is_v ? p.V : p.K) + w.b * st[0] + w.h * st[1] + w.t0 * step + 8 * lane8;
    uint4 v[kCacheRows];
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (u < w.n) v[u] = __ldg(reinterpret_cast<const uint4*>(src + u * step));
    }
    if constexpr (!E4M3) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.Vc : p.Kc) + w.at * D + 8 * lane8;
#pragma unroll
        for (int u = 0; u < kCacheRows; ++u)
            if (u < w.n) *reinterpret_cast<uint4*>(dst + u * D) = v[u];
    } else {
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.Vc : p.Kc) + w.at * D + 8 * lane8;
        uint8_t* dexp = (is_v ? p.ve : p.ke) + w.at;
        uint32_t top[kCacheRows / 2];  // largest magnitudes of two rows
#pragma unroll
        for (int u = 0; u < kCacheRows; u += 2) {
            uint32_t m[2];  // of the even and of the odd values of a row
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4& x = v[u + i];
                m[i] = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
            }
            top[u / 2] = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) {
#pragma unroll
            for (int u = 0; u < kCacheRows / 2; ++u) top[u] = __vmaxu2(top[u], __shfl_xor_sync(0xFFFFFFFFu, top[u], o));
        }
#pragma unroll
        for (int u = 0; u < kCacheRows; ++u) {
            const uint32_t t = (u & 1) ? top[u / 2] >> 16 : top[u / 2] & 0xFFFFu;
            // 1.m * 2^(E - 127) <= 1.75 * 2^8 * 2^(e - 127): the mantissas above 0x60 carry into E
            const bool bad = t >= 0x7F80u;
            const int e = bad ? 255 : max(1, static_cast<int>((t + 0x1Fu) >> 7) - 8);
            const float f = __uint_as_float(static_cast<uint32_t>(bad ? 127 : 254 - e) << 23);
            const uint64_t f2 = f2_pack(f, f);
            const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;
                f2_unpack(f2_mul(f2_pack(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xFFFF0000u)), f2), lo, hi);
                q[k] = e4m3x2(lo, hi);
            }
            if (u < w.n) {
                *reinterpret_cast<uint2*>(dst + u * D) =
                    bad ? make_uint2(0u, 0u) : make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
                if (lane8 == 0) dexp[u] = static_cast<uint8_t>(e);
            }
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheParams p) {
    constexpr int LPR = D / 8, G = kCacheThreads / LPR;
    const int lane8 = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const bool is_v = blockIdx.y != 0;
    const Segment w(p, blockIdx.x * G + group, (kKernCache << 8) | 0xB1u, lane8 == 0 && !is_v);
    __nv_bfloat16* out =
        (is_v ? p.Vo : p.Ko) + ((static_cast<int64_t>(w.b) * p.H + w.h) * p.tokens + w.t0) * D + 8 * lane8;
    if constexpr (!E4M3) {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.Vc : p.Kc) + w.at * D + 8 * lane8;
        uint4 v[kCacheRows];
#pragma unroll
        for (int u = 0; u < kCacheRows; ++u)
            if (u < w.n) v[u] = __ldg(reinterpret_cast<const uint4*>(src + u * D));
#pragma unroll
        for (int u = 0; u < kCacheRows; ++u)
            if (u < w.n) *reinterpret_cast<uint4*>(out + u * D) = v[u];
    } else {
        const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.Vc : p.Kc) + w.at * D + 8 * lane8;
        const uint8_t* sexp = (is_v ? p.ve : p.ke) + w.at;
        uint2 v[kCacheRows];
        uint32_t e[kCacheRows];
#pragma unroll
        for (int u = 0; u < kCacheRows; ++u) {
            if (u < w.n) {
                v[u] = __ldg(reinterpret_cast<const uint2*>(src + u * D));
                e[u] = __ldg(sexp + u);
            }
        }
#pragma unroll
        for (int u = 0; u < kCacheRows; ++u) {
            if (u >= w.n) break;
            const float f = exp_value(e[u]);
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t x = k < 2 ? v[u].x : v[u].y;
                const float2 y = (k & 1) ? e4m3x2_values<true>(x) : e4m3x2_values<false>(x);
                float lo, hi;
                f2_unpack(f2_mul(f2_pack(y.x, y.y), f2_pack(f, f)), lo, hi);
                o[k] = pack_bf16x2(lo, hi);
            }
            *reinterpret_cast<uint4*>(out + u * D) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Level-0 mean of one key block by one warp: D/16 lanes hold a row (16 bytes each), so a load
// instruction covers 32 / (D/16) rows; the loads of 32 keys are in flight together. Lane l holds the
// exponent of key l of every run of 32 and hands it round by shuffles. Every caller sums in this
// order, so appends equal builds bit for bit.
template <int D>
__device__ __forceinline__ void e4m3_block_mean(const uint8_t* K, const uint8_t* e, int blk, float* out) {
    constexpr int LPR = D / 16, RPI = 32 / LPR, N = 32 / RPI;
    const int lane = threadIdx.x & 31, chunk = lane % LPR, rsub = lane / LPR;
    uint64_t acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0ull;
    const uint8_t* row = K + rsub * D + 16 * chunk;
#pragma unroll 1
    for (int r0 = 0; r0 < blk; r0 += 32) {
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(row + (r0 + i * RPI) * D));
        const uint32_t ex = __ldg(e + r0 + lane);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float f = exp_value(__shfl_sync(0xFFFFFFFFu, ex, i * RPI + rsub));
            const uint64_t f2 = f2_pack(f, f);
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 x = (k & 1) ? e4m3x2_values<true>(w[k >> 1]) : e4m3x2_values<false>(w[k >> 1]);
                asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[k]) : "l"(f2_pack(x.x, x.y)), "l"(f2));
            }
        }
    }
    float a[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) f2_unpack(acc[k], a[2 * k], a[2 * k + 1]);
    // over the lanes of a chunk: each step two lanes share out what they hold, so a lane ends with 16 / RPI dims
    int at = 16 * chunk;
#pragma unroll
    for (int o = LPR, n = 8; o < 32; o <<= 1, n >>= 1) {
        const bool upper = (lane & o) != 0;
        at += upper ? n : 0;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float keep = upper ? a[n + k] : a[k], give = upper ? a[k] : a[n + k];
            a[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
    }
    const float inv = 1.0f / static_cast<float>(blk);
    if constexpr (RPI == 4)
        *reinterpret_cast<float4*>(out + at) = make_float4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
    else
        *reinterpret_cast<float2*>(out + at) = make_float2(a[0] * inv, a[1] * inv);
}

// Subtrees of S = f^m key blocks (S <= 16, or f): a CTA forms the level-0 means of its blocks that are
// new (one warp per block), takes the older ones as they stand, and forms the m levels above them in
// shared memory; nodes over older blocks alone come out as they were. Grid: planes x the subtrees
// that hold a new block.
template <int D>
__global__ void __launch_bounds__(256, 4) cache_subtree_kernel(const CachePyramidParams p, int S, int m, int sub_lo,
                                                            int subtrees) {
    extern __shared__ __align__(16) float rows[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t plane = blockIdx.x / subtrees;
    const int64_t j0 = static_cast<int64_t>(sub_lo + blockIdx.x % subtrees) * S;
    float* out = p.pyr + plane * p.plane_rows * D;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < S && j0 + r < p.n0; r += 8) {
        const int64_t j = j0 + r;
        float* row = rows + r * D;
        if (j >= p.b_lo) {
            const int64_t at = plane * p.N + j * p.blk;
            e4m3_block_mean<D>(p.K + at * D, p.e + at, p.blk, row);
            __syncwarp();
            for (int c = lane; c < D / 4; c += 32)
                reinterpret_cast<float4*>(out + j * D)[c] = reinterpret_cast<const float4*>(row)[c];
        } else {
            for (int c = lane; c < D / 4; c += 32)
                reinterpret_cast<float4*>(row)[c] = reinterpret_cast<const float4*>(out + j * D)[c];
        }
    }
    int64_t width = 1;
    int span = S;
    const float* below = rows;
    for (int l = 1; l <= m; ++l) {
        __syncthreads();
        const int up = span / p.factor;
        float* cur = rows + (below - rows) + span * D;
        const int64_t c0 = j0 / (width * p.factor), first = j0 / width;
        for (int e = threadIdx.x; e < up * (D / 4); e += 256) {
            const int64_t c = c0 + e / (D / 4);
            const int q = e % (D / 4);
            if (c >= p.lsize[l] || c * width * p.factor >= p.n0) continue;
            const float4 v = node_mean4(below + 4 * q, first, D, c, p.factor, p.lsize[l - 1], width, p.n0);
            *reinterpret_cast<float4*>(cur + (c - c0) * D + 4 * q) = v;
            *reinterpret_cast<float4*>(out + (p.loff[l] + c) * D + 4 * q) = v;
        }
        below = cur;
        span = up;
        width *= p.factor;
    }
}

// Level 0 of many new blocks without subtrees (a single level, or a factor above 64): one warp per block.
template <int D>
__global__ void __launch_bounds__(128) cache_block_mean_kernel(const CachePyramidParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int n = p.b_hi - p.b_lo;
    if (w >= static_cast<int64_t>(p.planes) * n) return;
    const int64_t plane = w / n;
    const int64_t j = p.b_lo + w % n;
    const int64_t row = plane * p.N + j * p.blk;
    e4m3_block_mean<D>(p.K + row * D, p.e + row, p.blk, p.pyr + (plane * p.plane_rows + j) * D);
}

// The nodes of levels l0 .. L - 1 over the blocks [b_lo, b_hi) of one plane per CTA, level after level.
template <int D>
__global__ void __launch_bounds__(256) cache_pyramid_kernel(const CachePyramidParams p, int l0) {
    const int64_t plane = blockIdx.x;
    float* out = p.pyr + plane * p.plane_rows * D;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the grid before is complete
    int64_t width = 1;
    for (int l = 1; l < l0; ++l) width *= p.factor;
    for (int l = l0; l < p.L; ++l) {
        __syncthreads();
        const int64_t wl = width * p.factor;
        const int c_lo = static_cast<int>(p.b_lo / wl);
        const int c_hi = static_cast<int>(min(static_cast<int64_t>(p.lsize[l]), (p.b_hi - 1) / wl + 1));
        const float* below = out + static_cast<int64_t>(p.loff[l - 1]) * D;
        for (int e = threadIdx.x; e < (c_hi - c_lo) * (D / 4); e += blockDim.x) {
            const int c = c_lo + e / (D / 4), q = e % (D / 4);
            *reinterpret_cast<float4*>(out + (static_cast<int64_t>(p.loff[l]) + c) * D + 4 * q) =
                node_mean4(below + 4 * q, 0, D, c, p.factor, p.lsize[l - 1], width, p.n0);
        }
        width = wl;
    }
}

// A whole append of few blocks in one launch, one plane per CTA. What is older than the append and still
// counts, the siblings to the left of the first new node of every level, is fetched into shared memory
// while the level-0 means are formed, so the levels above follow from shared memory alone. `lo[l]`: first
// row of level l held (the first new node's leftmost sibling), `at[l]`: where its rows begin.
struct AppendRows {
    int32_t lo[PISA_MAX_LEVELS], hi[PISA_MAX_LEVELS], fresh[PISA_MAX_LEVELS], at[PISA_MAX_LEVELS];
};
template <int D>
__global__ void __launch_bounds__(256) cache_append_kernel(const CachePyramidParams p, const AppendRows a) {
    extern __shared__ __align__(16) float rows[];
    const int64_t plane = blockIdx.x;
    float* out = p.pyr + plane * p.plane_rows * D;
    const int warp = threadIdx.x >> 5;
    for (int l = 0; l < p.L; ++l) {
        for (int e = threadIdx.x; e < (a.fresh[l] - a.lo[l]) * (D / 4); e += blockDim.x)
            reinterpret_cast<float4*>(rows + a.at[l] * D)[e] =
                reinterpret_cast<const float4*>(out + (static_cast<int64_t>(p.loff[l]) + a.lo[l]) * D)[e];
    }
    for (int j = p.b_lo + warp; j < p.b_hi; j += blockDim.x >> 5) {
        const int64_t at = plane * p.N + static_cast<int64_t>(j) * p.blk;
        e4m3_block_mean<D>(p.K + at * D, p.e + at, p.blk, rows + (a.at[0] + j - a.lo[0]) * D);
    }
    int64_t width = 1;
    for (int l = 0; l < p.L; ++l) {
        __syncthreads();
        const int n = a.hi[l] - a.fresh[l];
        float* level = rows + a.at[l] * D;
        float* dst = out + (static_cast<int64_t>(p.loff[l]) + a.fresh[l]) * D;
        for (int e = threadIdx.x; e < n * (D / 4); e += blockDim.x) {
            const int c = a.fresh[l] + e / (D / 4), q = e % (D / 4);
            float4 v;
            if (l == 0) {
                v = *reinterpret_cast<const float4*>(level + (c - a.lo[0]) * D + 4 * q);
            } else {
                v = node_mean4(rows + a.at[l - 1] * D + 4 * q, a.lo[l - 1], D, c, p.factor, p.lsize[l - 1], width, p.n0);
                *reinterpret_cast<float4*>(level + (c - a.lo[l]) * D + 4 * q) = v;
            }
            reinterpret_cast<float4*>(dst)[e] = v;
        }
        if (l > 0) width *= p.factor;
    }
}

template <int D>
static bool launch_cache_rows(const CacheParams& p, bool e4m3, bool write, cudaStream_t st) {
    constexpr int G = kCacheThreads / (D / 8);
    const int64_t segments = static_cast<int64_t>(p.B) * p.H * ((p.tokens + kCacheRows - 1) / kCacheRows);
    const int64_t blocks = (segments + G - 1) / G;
    if (blocks > INT32_MAX) return false;
    const dim3 grid(static_cast<unsigned>(blocks), 2);
    if (write) {
        if (e4m3)
            cache_write_kernel<D, true><<<grid, kCacheThreads, 0, st>>>(p);
        else
            cache_write_kernel<D, false><<<grid, kCacheThreads, 0, st>>>(p);
    } else {
        if (e4m3)
            cache_read_kernel<D, true><<<grid, kCacheThreads, 0, st>>>(p);
        else
            cache_read_kernel<D, false><<<grid, kCacheThreads, 0, st>>>(p);
    }
    return cudaGetLastError() == cudaSuccess;
}

bool launch_cache_write(const CacheParams& p, int D, bool e4m3, cudaStream_t st) {
    return D == 64 ? launch_cache_rows<64>(p, e4m3, true, st) : launch_cache_rows<128>(p, e4m3, true, st);
}

bool launch_cache_read(const CacheParams& p, int D, bool e4m3, cudaStream_t st) {
    return D == 64 ? launch_cache_rows<64>(p, e4m3, false, st) : launch_cache_rows<128>(p, e4m3, false, st);
}

// New blocks per plane up to which an append is one launch (a plane's 8 warps take one block each), if the
// rows it holds fit this much shared memory; past it the level-0 means get a grid of their own, whose
// warps fill the SMs. (One new block in 64 x 8 planes of 256 blocks: 11.4 us when every level read the one
// below from global memory.)
constexpr int kCachePyramidOneLaunch = 8;
constexpr size_t kCacheAppendSmem = 48 * 1024;

template <int D>
static bool launch_cache_pyramid_d(const CachePyramidParams& p, cudaStream_t st, int32_t* launches) {
    if (p.b_hi - p.b_lo <= kCachePyramidOneLaunch) {
        AppendRows a{};
        int64_t total = 0, width = 1;
        for (int l = 0; l < p.L; ++l) {
            a.fresh[l] = static_cast<int32_t>(p.b_lo / width);
            a.hi[l] = static_cast<int32_t>((p.b_hi - 1) / width + 1);
            a.lo[l] = l + 1 < p.L ? a.fresh[l] / p.factor * p.factor : a.fresh[l];
            a.at[l] = static_cast<int32_t>(total);
            total += a.hi[l] - a.lo[l];
            width *= p.factor;
        }
        if (total * D * sizeof(float) <= kCacheAppendSmem) {
            // a warp per new block, two at least: many planes of one block each then fit the SMs at once
            const int threads = p.b_hi - p.b_lo <= 2 ? 64 : 256;
            cache_append_kernel<D><<<p.planes, threads, total * D * sizeof(float), st>>>(p, a);
            if (cudaGetLastError() != cudaSuccess) return false;
            ++*launches;
            return true;
        }
    }
    int l0 = 1;  // first level that the second launch forms
    if (p.L >= 2 && p.factor <= 64) {
        int S = p.factor, m = 1;
        while (m + 1 <= p.L - 1 && S * p.factor <= 16) {
            S *= p.factor;
            ++m;
        }
        int rows = 0, span = S;
        for (int l = 0; l <= m; ++l, span /= p.factor) rows += span;
        const int sub_lo = p.b_lo / S, subtrees = (p.b_hi - 1) / S + 1 - sub_lo;
        const int64_t blocks = static_cast<int64_t>(p.planes) * subtrees;
        if (blocks > INT32_MAX) return false;
        cache_subtree_kernel<D><<<static_cast<unsigned>(blocks), 256, rows * D * sizeof(float), st>>>(p, S, m, sub_lo,
                                                                                                      subtrees);
        l0 = m + 1;
    } else {
        const int64_t warps = static_cast<int64_t>(p.planes) * (p.b_hi - p.b_lo);
        if ((warps + 3) / 4 > INT32_MAX) return false;
        cache_block_mean_kernel<D><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, st>>>(p);
    }
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    if (l0 >= p.L) return true;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.planes));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, cache_pyramid_kernel<D>, p, l0) != cudaSuccess) return false;
    ++*launches;
    return true;
}

bool launch_cache_pyramid(const CachePyramidParams& p, cudaStream_t st, int32_t* launches) {
    return p.D == 64 ? launch_cache_pyramid_d<64>(p, st, launches) : launch_cache_pyramid_d<128>(p, st, launches);
}

}  // namespace pisa
