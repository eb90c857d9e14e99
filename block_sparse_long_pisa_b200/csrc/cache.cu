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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pisa_device.cuh"
#include "pisa_pool.cuh"

namespace pisa {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 4;  // rows one lane group has in flight

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 e4m3x2_values(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// 2^(e - 127) of an exponent byte 1 .. 254; 255 gives an infinity, which times a zero byte is the
// NaN that such a row stands for.
__device__ __forceinline__ float exp_value(uint32_t e) { return __uint_as_float(e << 23); }

// The sequence's first cache position and row count; false when the range does not fit the cache.
__device__ __forceinline__ bool cache_range(const CacheParams& p, int b, int64_t& start, int& count) {
    start = p.start != nullptr ? p.start[b] : 0;
    count = p.count != nullptr ? p.count[b] : p.tokens;
    return count >= 0 && count <= p.tokens && start >= 0 && start + count <= p.cap;
}

// Row r of the call -> sequence, head, token (tokens fastest).
struct RowAt {
    int b, h, t;
    __device__ __forceinline__ RowAt(const CacheParams& p, uint32_t r) {  // B * H * tokens < 2^31
        const uint32_t q = r / static_cast<uint32_t>(p.tokens);
        t = static_cast<int>(r - q * static_cast<uint32_t>(p.tokens));
        b = static_cast<int>(q / static_cast<uint32_t>(p.H));
        h = static_cast<int>(q - static_cast<uint32_t>(b) * static_cast<uint32_t>(p.H));
    }
};

// grid: (row blocks, K or V). Each lane group takes kCacheRows rows, a block's groups side by side.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
    constexpr int LPR = D / 8, G = kCacheThreads / LPR;
    const int lane8 = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const bool is_v = blockIdx.y != 0;
    const uint32_t rows = static_cast<uint32_t>(p.B) * p.H * p.tokens;
    const uint32_t r0 = blockIdx.x * (G * kCacheRows) + group;
    const __nv_bfloat16* src = is_v ? p.V : p.K;
    const int64_t s0 = is_v ? p.vs[0] : p.ks[0], s1 = is_v ? p.vs[1] : p.ks[1], s2 = is_v ? p.vs[2] : p.ks[2];
    uint4 v[kCacheRows];
    int64_t at[kCacheRows];
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
        const uint32_t r = r0 + u * G;
        at[u] = -1;
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= rows) continue;
        const RowAt w(p, r);
        int64_t start;
        int count;
        if (!cache_range(p, w.b, start, count)) {
            if (lane8 == 0 && w.h == 0 && w.t == 0 && !is_v)
                record_error(p.status, PISA_ERR_BAD_INDEX, (kKernCache << 8) | 0xB0u);
            continue;
        }
        if (w.t >= count) continue;
        at[u] = (static_cast<int64_t>(w.b) * p.H + w.h) * p.cap + start + w.t;
        v[u] = __ldg(reinterpret_cast<const uint4*>(src + w.b * s0 + w.h * s1 + w.t * s2 + 8 * lane8));
    }
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
        if constexpr (!E4M3) {
            if (at[u] >= 0)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.Vc : p.Kc) + at[u] * D + 8 * lane8) =
                    v[u];
        } else {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            uint32_t top = 0;  // largest magnitude of the even and of the odd values
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            top = max(top & 0xFFFFu, top >> 16);
            // 1.m * 2^(E - 127) <= 1.75 * 2^8 * 2^(e - 127)
            const int E = static_cast<int>(top >> 7);
            const bool bad = E == 255;
            const int e = bad ? 255 : max(1, E - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0));
            const float f = __uint_as_float(static_cast<uint32_t>(bad ? 127 : 254 - e) << 23);
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                q[k] = e4m3x2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
            if (at[u] >= 0) {
                uint8_t* dst = static_cast<uint8_t*>(is_v ? p.Vc : p.Kc) + at[u] * D + 8 * lane8;
                *reinterpret_cast<uint2*>(dst) =
                    bad ? make_uint2(0u, 0u) : make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
                if (lane8 == 0) (is_v ? p.ve : p.ke)[at[u]] = static_cast<uint8_t>(e);
            }
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheParams p) {
    constexpr int LPR = D / 8, G = kCacheThreads / LPR;
    const int lane8 = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const bool is_v = blockIdx.y != 0;
    const uint32_t rows = static_cast<uint32_t>(p.B) * p.H * p.tokens;
    const uint32_t r0 = blockIdx.x * (G * kCacheRows) + group;
    __nv_bfloat16* out = is_v ? p.Vo : p.Ko;
    uint4 v[kCacheRows];
    uint32_t e[kCacheRows];
    bool ok[kCacheRows];
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
        const uint32_t r = r0 + u * G;
        ok[u] = false;
        if (r >= rows) continue;
        const RowAt w(p, r);
        int64_t start;
        int count;
        if (!cache_range(p, w.b, start, count)) {
            if (lane8 == 0 && w.h == 0 && w.t == 0 && !is_v)
                record_error(p.status, PISA_ERR_BAD_INDEX, (kKernCache << 8) | 0xB1u);
            continue;
        }
        if (w.t >= count) continue;
        ok[u] = true;
        const int64_t at = (static_cast<int64_t>(w.b) * p.H + w.h) * p.cap + start + w.t;
        if constexpr (E4M3) {
            const uint2 two = __ldg(reinterpret_cast<const uint2*>(
                static_cast<const uint8_t*>(is_v ? p.Vc : p.Kc) + at * D + 8 * lane8));
            v[u].x = two.x;
            v[u].y = two.y;
            e[u] = __ldg((is_v ? p.ve : p.ke) + at);
        } else {
            v[u] = __ldg(reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(is_v ? p.Vc : p.Kc) + at * D + 8 * lane8));
        }
    }
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
        if (!ok[u]) continue;
        if constexpr (E4M3) {
            const float f = exp_value(e[u]);
            const uint32_t w[2] = {v[u].x, v[u].y};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = e4m3x2_values((w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
                o[k] = pack_bf16x2(x.x * f, x.y * f);
            }
            v[u] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r0 + u * G) * D + 8 * lane8) = v[u];
    }
}

// Level-0 mean of one key block by one warp: D/16 lanes hold a row (16 bytes each), so a load
// instruction covers 32 / (D/16) rows; the warp's loads of a 64-key block are all in flight
// together. Lane l holds the exponents of keys l and l + 32 of every run of 64 and hands them round
// by shuffles. Every caller sums in this order, so appends equal builds bit for bit.
template <int D>
__device__ __forceinline__ void e4m3_block_mean(const uint8_t* K, const uint8_t* e, int blk, float* out) {
    constexpr int LPR = D / 16, RPI = 32 / LPR, N = 64 / RPI;
    const int lane = threadIdx.x & 31, chunk = lane % LPR, rsub = lane / LPR;
    float acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    for (int r0 = 0; r0 < blk; r0 += 64) {
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = __ldg(reinterpret_cast<const uint4*>(K + static_cast<int64_t>(r0 + i * RPI + rsub) * D) + chunk);
        const uint32_t e0 = __ldg(e + r0 + lane), e1 = __ldg(e + r0 + 32 + lane);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = i * RPI + rsub;
            const float f = exp_value(__shfl_sync(0xFFFFFFFFu, i * RPI < 32 ? e0 : e1, row & 31));
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 x = e4m3x2_values((w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
                acc[2 * k] = fmaf(x.x, f, acc[2 * k]);
                acc[2 * k + 1] = fmaf(x.y, f, acc[2 * k + 1]);
            }
        }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] += __shfl_xor_sync(0xFFFFFFFFu, acc[k], o);
    }
    if (rsub == 0) {
        const float inv = 1.0f / static_cast<float>(blk);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            reinterpret_cast<float4*>(out + 16 * chunk)[k] = make_float4(acc[4 * k] * inv, acc[4 * k + 1] * inv,
                                                                         acc[4 * k + 2] * inv, acc[4 * k + 3] * inv);
    }
}

// Level 0 of many new blocks: one warp per block.
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

// The nodes over the blocks [b_lo, b_hi) of one plane per CTA, level after level; with LEVEL0 (few
// new blocks) the CTA's warps form the level-0 means first, and the whole append is one launch.
template <int D, bool LEVEL0>
__global__ void __launch_bounds__(256) cache_pyramid_kernel(const CachePyramidParams p) {
    const int64_t plane = blockIdx.x;
    float* out = p.pyr + plane * p.plane_rows * D;
    if constexpr (LEVEL0) {
        for (int j = p.b_lo + (threadIdx.x >> 5); j < p.b_hi; j += blockDim.x >> 5) {
            const int64_t row = plane * p.N + static_cast<int64_t>(j) * p.blk;
            e4m3_block_mean<D>(p.K + row * D, p.e + row, p.blk, out + static_cast<int64_t>(j) * D);
        }
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the level-0 grid is complete
    }
    int64_t width = 1;
    for (int l = 1; l < p.L; ++l) {
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

template <int D>
static bool launch_cache_rows(const CacheParams& p, bool e4m3, bool write, cudaStream_t st) {
    constexpr int per_block = kCacheThreads / (D / 8) * kCacheRows;
    const int64_t rows = static_cast<int64_t>(p.B) * p.H * p.tokens;
    const int64_t blocks = (rows + per_block - 1) / per_block;
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

// New blocks per plane up to which an append is one launch (a plane's 8 warps take one block each);
// past it the level-0 means get a grid of their own, whose warps fill the SMs.
constexpr int kCachePyramidOneLaunch = 8;

template <int D>
static bool launch_cache_pyramid_d(const CachePyramidParams& p, cudaStream_t st, int32_t* launches) {
    if (p.b_hi - p.b_lo <= kCachePyramidOneLaunch) {
        cache_pyramid_kernel<D, true><<<p.planes, 256, 0, st>>>(p);
        if (cudaGetLastError() != cudaSuccess) return false;
        ++*launches;
        return true;
    }
    const int64_t warps = static_cast<int64_t>(p.planes) * (p.b_hi - p.b_lo);
    cache_block_mean_kernel<D><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return false;
    ++*launches;
    if (p.L < 2) return true;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.planes));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, cache_pyramid_kernel<D, false>, p) != cudaSuccess) return false;
    ++*launches;
    return true;
}

bool launch_cache_pyramid(const CachePyramidParams& p, cudaStream_t st, int32_t* launches) {
    return p.D == 64 ? launch_cache_pyramid_d<64>(p, st, launches) : launch_cache_pyramid_d<128>(p, st, launches);
}

}  // namespace pisa
