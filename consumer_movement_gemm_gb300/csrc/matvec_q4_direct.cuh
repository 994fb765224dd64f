// matvec_q4_direct.cuh -- 4-bit products whose time is latency: no ring, no
// workspace, no counter.  A CTA takes 32 columns; its warps take every 8th or
// 16th block of 128 rows, straight from global memory into registers (a block
// ahead of the one that is multiplied, and the same products as in skinny.cuh);
// the warps' sums meet once in shared memory, in the order of the warps.  Where
// there are few columns, a cluster of two or four CTAs shares out the rows, and
// its first CTA gets the others' sums through distributed shared memory.
//
// What it costs: the rows of the activations come from L2 once per 32 columns
// and lane (the ring stages them once per 512 columns), and a CTA's first loads
// and its join are bare.  What bounds it: the dependent loads of a CTA, launch to
// store, at small sizes (512 x 512: 1.9 us, 2048 x 2048: 3.2, 4096 x 4096: 4.9
// with one row, where the ring takes 7.6, 7.6 and 8.4), the loads in flight at
// large ones (3.1 TB/s with one row, the ring 4.0).
#pragma once
#include "skinny.cuh"

namespace tovl {
namespace skinny {

constexpr int kDirectWarps = 16;              // at most; CTAs of 8 share an SM
constexpr int kDirectCols = 32;
constexpr int kDirectCluster = 4;

// What a lane holds of a block: words, scales and zeros of its four columns,
// and its octets of the rows.
template <int NT, bool XS, int G, bool Z>
struct DirectBlock {
    static constexpr int kGroups = 128 / G;
    uint4 w[4], x[4][NT];
    uint2 scale[kGroups];
    uint32_t zero[kGroups];
    float xs[NT];

    __device__ __forceinline__ void load_weights(const MatvecDirectParams& p, int b, int n, bool col, int t)
    {
#pragma unroll
        for (int R = 0; R < 4; ++R) {
            const int octet = b * 16 + 4 * R + t;
            w[R] = make_uint4(0, 0, 0, 0);
            if (col && octet * 8 < p.K) w[R] = ld_stream(static_cast<const uint32_t*>(p.wq) + static_cast<long long>(octet) * p.N + n);
        }
    }
    __device__ __forceinline__ void load_scales(const MatvecDirectParams& p, int b, int n, bool col)
    {
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            const bool in = col && b * 128 + q * G < p.K;
            const long long at = (static_cast<long long>(b) * kGroups + q) * p.N + n;
            scale[q] = in ? __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.w_scale) + at)) : make_uint2(0, 0);
            zero[q] = Z && in ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.w_zero) + at)) : 0u;
        }
    }
    // as they are in memory; a row past the last one repeats the first, its result is not stored
    __device__ __forceinline__ void load_rows(const MatvecDirectParams& p, int b, int r0, int cnt, int g, int t)
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const long long row = r0 + (nt * 8 + g < cnt ? nt * 8 + g : 0);
#pragma unroll
            for (int R = 0; R < 4; ++R) {
                const int k = b * 128 + 32 * R + 8 * t;
                x[R][nt] = make_uint4(0, 0, 0, 0);
                if (k >= p.K) continue;
                if (XS) {
                    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x) + row * p.ldx + k));
                    x[R][nt].x = u.x;
                    x[R][nt].y = u.y;
                } else {
                    x[R][nt] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + row * p.ldx + k));
                }
            }
            if (XS) xs[nt] = __ldg(p.x_scale + row * ((p.K + kXScaleGroup - 1) / kXScaleGroup) + b);
        }
    }
    // to fp16, and the scales of the tokens of this lane's sums (2 t, 2 t + 1)
    __device__ __forceinline__ void convert_rows(float2 (&sx)[NT], int t)
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float own;
            if (XS) {
#pragma unroll
                for (int R = 0; R < 4; ++R) {
                    const uint2 lo = e4m3x4_to_half(x[R][nt].x), hi = e4m3x4_to_half(x[R][nt].y);
                    x[R][nt] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
                own = xs[nt];
            } else {
                uint32_t e = 0;
#pragma unroll
                for (int R = 0; R < 4; ++R) e = max(e, max_exponent(x[R][nt]));
                e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
                e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
                const float f = half_scale(e);
#pragma unroll
                for (int R = 0; R < 4; ++R) x[R][nt] = bf16x8_to_half(x[R][nt], f);
                own = half_unscale(e);
            }
            sx[nt].x = __shfl_sync(0xffffffffu, own, 8 * t);
            sx[nt].y = __shfl_sync(0xffffffffu, own, 8 * t + 4);
        }
    }
};

template <int NT, bool XS, int G, bool Z>
__global__ void __launch_bounds__(kDirectWarps * 32, 1) matvec_q4_direct_kernel(const __grid_constant__ MatvecDirectParams p)
{
    // (columns in fours, the four of token r exchanged by r / 2: no bank conflicts)
    __shared__ __align__(16) float red[kDirectWarps][NT * 8][kDirectCols];
    __shared__ float join[kDirectCluster - 1][NT * 8][kDirectCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5, split = gridDim.y, rank = blockIdx.y;      // the cluster: CTAs (1, split, 1)
    const int r0 = blockIdx.z * 16, cnt = min(16, p.T - r0);
    const int n = blockIdx.x * kDirectCols + 4 * column_group(g);
    const bool col = n < p.N;                 // (N is a multiple of 8: four columns are in or out together)
    const int blocks = (p.K + 127) / 128, stride = warps * split;
    if (split > 1) ptx::cluster_arrive_relaxed();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    float acc[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;

    using Block = DirectBlock<NT, XS, G, Z>;
    constexpr bool kAllAhead = NT == 1;       // two rows' tiles of the next block would not fit the registers
    int b = rank * warps + warp;
    Block next;
    const auto fetch_weights = [&](int at) {
        next.load_weights(p, at, n, col, t);
        if (kAllAhead) {
            next.load_scales(p, at, n, col);
            next.load_rows(p, at, r0, cnt, g, t);
        }
    };
    if (b < blocks) fetch_weights(b);
    for (; b < blocks; b += stride) {
        Block now = next;
        if (!kAllAhead) {
            now.load_scales(p, b, n, col);
            now.load_rows(p, b, r0, cnt, g, t);
        }
        if (b + stride < blocks) fetch_weights(b + stride);
        float2 sx[NT];
        now.convert_rows(sx, t);
        multiply_q4<NT, G, Z>(
            acc, sx, [&](int R) { return now.w[R]; }, [&](int q) { return now.zero[q]; }, [&](int q) { return now.scale[q]; },
            [&](int R, int nt) { return now.x[R][nt]; });
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<float4*>(&red[warp][nt * 8 + 2 * t + j][4 * (column_group(g) ^ t)]) =
                make_float4(acc[0][nt][j], acc[0][nt][j + 2], acc[1][nt][j], acc[1][nt][j + 2]);
    __syncthreads();
    // sums of row r of column c: a warp each, 8 or 16 rows at a time
    const int c = threadIdx.x & 31, at = blockIdx.x * kDirectCols + c;
    if (split > 1) {
        __syncwarp();
        ptx::cluster_wait();                  // the first CTA of the cluster runs
    }
    const auto sum = [&](int r) {
        float v = 0.f;
        const int at = c ^ ((r >> 1 & 3) << 2);
#pragma unroll
        for (int i = 0; i < kDirectWarps / 2; ++i) v += red[i][r][at];
        if (warps > kDirectWarps / 2) {
#pragma unroll
            for (int i = kDirectWarps / 2; i < kDirectWarps; ++i) v += red[i][r][at];
        }
        return v;
    };
    if (split > 1) {
        if (rank > 0)
            for (int r = warp; r < cnt; r += warps) st_cluster_f32(ptx::mapa_shared(ptx::smem_u32(&join[rank - 1][r][c]), 0), sum(r));
        __syncwarp();
        ptx::cluster_sync();
        if (rank > 0) return;
    }
    for (int r = warp; r < cnt; r += warps) {
        float v = sum(r);
        for (int i = 1; i < split; ++i) v += join[i - 1][r][c];
        if (at < p.N) static_cast<__nv_bfloat16*>(p.out)[(r0 + r) * p.ldo + at] = __float2bfloat16(v);
    }
}

}  // namespace skinny
}  // namespace tovl
