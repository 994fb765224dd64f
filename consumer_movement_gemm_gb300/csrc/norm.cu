// norm.cu -- residual addition and root-mean-square norm of token rows, with
// a bf16 output and an e4m3 output that has one fp32 scale per group.
//
//   r = x + residual            y = r * rsqrt(mean(r^2) + eps) * weight
//   residual_out = round(r)     out = bf16(y)
//   scale = max(amax over the group of |y|, 1e-12) / 448,   q = e4m3(y / scale)
//
// One pass over memory: a row stays in registers from the load to the last
// store, everything is fp32 in between.  Rows up to 1024 elements take a warp
// each (no barrier), longer ones a CTA each (one barrier a reduction).  A thread holds
// groups of 8 consecutive elements, so a scale group of 32, 64 or 128 columns
// is 4, 8 or 16 neighbouring lanes.
//
// What bounds it: memory.  Rows of whole 16-byte pieces (norm_rows_kernel): 16384 x
// 7168, bf16 residual, both outputs, 167 us, 6.3 TB/s; 16384 x 8192 203 us, 6.0;
// 333 x 7168, fp32 residual, 8.3 us (one to three rows an SM: their latency); 1 x
// 4096 2.7 us.  Rows that start elsewhere: norm_offset_kernel, norm_kernel.
#include <cuda_bf16.h>
#include <type_traits>
#include "common.cuh"
#include "ops.cuh"

namespace tovl {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinAmax = 1e-12f;     // keeps 448 / amax finite
constexpr int kWarpRows = 8;           // rows per CTA of the warp-per-row form
constexpr int kWarpRowMax = 1024;      // longest row of the warp-per-row form
constexpr int kOffsetThreads = 1024;   // at most, of a CTA whose rows start off the boundaries

// Larger operand, NaN if one is (a NaN shows in its group's scale).
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// A group's scale and what its elements' quotients by it are made with.  A product
// with 448 / max rounds twice, and its e4m3 is the wrong neighbour where y / scale
// lies half way between two, as 175 / 7 does; one residual of the fused
// multiply-add takes the quotient to 2^-46 before its own rounding (Markstein 1990,
// "Computation of elementary functions on the IBM RISC System/6000 processor").
// 16384 x 7168: 167 us with the residual, 172 with the product alone, 186 with a
// division; off the boundaries (16384 x 777) 45.5, 43.5 and 53.
struct Scale {
    float s, inverse;
    __device__ __forceinline__ explicit Scale(float amax) : s(max_nan(amax, kMinAmax) / kE4m3Max), inverse(1.f / s) {}
    __device__ __forceinline__ explicit Scale(float2 of) : s(of.x), inverse(of.y) {}
    __device__ __forceinline__ float divide(float y) const
    {
        // (an infinite scale: no residual, the quotients are 0, or NaN of an infinity; -0
        // gives +0)
        const float q = y * inverse;
        return fmaf(fmaf(-q, s == INFINITY ? 0.f : s, y), inverse, q);
    }
};

// Eight consecutive elements, of which the first n exist, moved in accesses of
// W elements.
template <int W>
__device__ __forceinline__ void load8(float (&v)[8], const __nv_bfloat16* p, int n)
{
    if constexpr (W == 8) {
        if (n <= 0) return;
        const uint4 u = __ldcg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else if constexpr (W == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * i < n) {
                const float2 f = unpack2(__ldcg(reinterpret_cast<const uint32_t*>(p) + i));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i] = __bfloat162float(p[i]);
    }
}

template <int W>
__device__ __forceinline__ void load8(float (&v)[8], const float* p, int n)
{
    if constexpr (W == 8) {
        if (n <= 0) return;
        const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i] = __ldcg(p + i);
    }
}

template <int W>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8], int n)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ptx::pack_bf16x2(v[2 * i], v[2 * i + 1]);
    if constexpr (W == 8) {
        if (n > 0) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (W == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * i < n) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = __float2bfloat16(v[i]);
    }
}

template <int W>
__device__ __forceinline__ void store8(float* p, const float (&v)[8], int n)
{
    if constexpr (W == 8) {
        if (n <= 0) return;
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

template <int W>
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&v)[8], const Scale& scale, int n)
{
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = e4m3x2(scale.divide(v[2 * i]), scale.divide(v[2 * i + 1]));
    if constexpr (W == 8) {
        if (n > 0) *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    } else if constexpr (W == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * i < n) reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(h[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = static_cast<uint8_t>(h[i / 2] >> (8 * (i & 1)));
    }
}

// Sum (or NaN-keeping maximum) over the threads of a row; every thread gets
// the same value, added in the same order.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* buf, bool warp_row)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, d);
        v = MAX ? max_nan(v, o) : v + o;
    }
    if (warp_row) return v;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? buf[lane] : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, d);
        v = MAX ? max_nan(v, o) : v + o;
    }
    return v;
}

// e4m3 of eight elements from column c on in a group of 32, 64 or 128 columns
// (4, 8 or 16 neighbouring lanes; whole warps call it).
template <int W>
__device__ __forceinline__ void store_group(const NormParams& p, int c, const float (&v)[8], float m, float* scale, uint8_t* q)
{
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (p.group > 32) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 4));
    if (p.group > 64) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
    const Scale of(m);
    if (c % p.group == 0 && c < p.H) scale[c / p.group] = of.s;
    store8_e4m3<W>(q + c, v, of, p.H - c);
}

// Sixteen-byte pieces of a row as they come from memory.
template <int RES>
struct Raw {
    uint4 x, r0, r1;      // r1: fp32 residuals only
};

__device__ __forceinline__ void unpack8(float (&v)[8], const uint4& u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// Rows of whole 16-byte pieces.  Every CTA (or warp, WARP) goes through rows a
// grid apart; the next row's loads are issued before this row is reduced, so
// the memory system never waits for the reduction, and the weights stay in
// registers.  RES: 0 none, 1 bf16, 2 fp32.  VPT: groups of 8 elements per
// thread.
template <int VPT, int RES, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpRows * 32 : 512, VPT <= 2 ? 2 : 1) norm_rows_kernel(const NormParams p)
{
    __shared__ float sum_buf[2][32], max_buf[2][32];
    const long long rows_step = static_cast<long long>(gridDim.x) * (WARP ? kWarpRows : 1);
    long long row = WARP ? static_cast<long long>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int step = (WARP ? 32 : blockDim.x) * 8;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (row >= p.T) return;     // whole warps (WARP), or whole CTAs
    uint4 weight[VPT];
    Raw<RES> next[VPT];
    // (not through the read-only path: the outputs may lie where the inputs do)
    const auto fetch = [&](long long r) {
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + r * p.ldx;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid * 8 + j * step;
            next[j].x = next[j].r0 = next[j].r1 = make_uint4(0, 0, 0, 0);
            if (c >= p.H) continue;
            next[j].x = __ldcg(reinterpret_cast<const uint4*>(x + c));
            if (RES == 1) next[j].r0 = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.residual) + r * p.ldr + c));
            if (RES == 2) {
                const uint4* f = reinterpret_cast<const uint4*>(static_cast<const float*>(p.residual) + r * p.ldr + c);
                next[j].r0 = __ldcg(f);
                next[j].r1 = __ldcg(f + 1);
            }
        }
    };
    fetch(row);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = tid * 8 + j * step;
        weight[j] = make_uint4(0, 0, 0, 0);
        if (c < p.H) weight[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.weight) + c));
    }
    for (int turn = 0; row < p.T; row += rows_step, turn ^= 1) {
        float v[VPT][8], ss = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid * 8 + j * step;
            unpack8(v[j], next[j].x);
            if (RES == 1) {
                float o[8];
                unpack8(o, next[j].r0);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] += o[i];
                store8<8>(static_cast<__nv_bfloat16*>(p.residual_out) + row * p.ldr + c, v[j], p.H - c);
            }
            if (RES == 2) {
                const uint32_t o[8] = {next[j].r0.x, next[j].r0.y, next[j].r0.z, next[j].r0.w,
                                       next[j].r1.x, next[j].r1.y, next[j].r1.z, next[j].r1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] += __uint_as_float(o[i]);
                store8<8>(static_cast<float*>(p.residual_out) + row * p.ldr + c, v[j], p.H - c);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
        }
        if (row + rows_step < p.T) fetch(row + rows_step);
        ss = row_reduce<false>(ss, sum_buf[turn], WARP);
        const float inv_rms = rsqrtf(ss / p.H + p.eps);
        float amax[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float g[8];
            unpack8(g, weight[j]);
            amax[j] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][i] = v[j][i] * inv_rms * g[i];
                amax[j] = max_nan(amax[j], fabsf(v[j][i]));
            }
            const int c = tid * 8 + j * step;
            if (c >= p.H) amax[j] = 0.f;       // (zeros times an infinite 1 / rms)
            if (p.out) store8<8>(static_cast<__nv_bfloat16*>(p.out) + row * p.ldo + c, v[j], p.H - c);
        }
        if (!p.q) continue;
        float* scale = p.q_scale + row * p.n_groups;
        uint8_t* q = p.q + row * p.H;
        if (p.group == p.H) {
            float m = amax[0];
#pragma unroll
            for (int j = 1; j < VPT; ++j) m = max_nan(m, amax[j]);
            const Scale of(row_reduce<true>(m, max_buf[turn], WARP));
            if (tid == 0) scale[0] = of.s;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = tid * 8 + j * step;
                store8_e4m3<8>(q + c, v[j], of, p.H - c);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPT; ++j) store_group<8>(p, tid * 8 + j * step, v[j], amax[j], scale, q);
        }
    }
}

// Rows of any length and alignment, moved in pairs or single elements (W = 8:
// whole pieces, for rows too long for a second one in the registers).
template <int W, int VPT, int RES>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p, int warp_row)
{
    __shared__ float sum_buf[32], max_buf[32];
    using R = typename std::conditional<RES == 2, float, __nv_bfloat16>::type;
    const long long row = warp_row ? static_cast<long long>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = warp_row ? threadIdx.x & 31 : threadIdx.x;
    const int step = (warp_row ? 32 : blockDim.x) * 8;
    const __nv_bfloat16* weight = static_cast<const __nv_bfloat16*>(p.weight);
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (row >= p.T) return;     // whole warps only
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + row * p.ldx;
    float v[VPT][8], g[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = tid * 8 + j * step;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = g[j][i] = 0.f;
        load8<W>(v[j], x + c, p.H - c);
        load8<W>(g[j], weight + c, p.H - c);
    }
    if (RES) {
        const R* res = static_cast<const R*>(p.residual) + row * p.ldr;
        float o[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid * 8 + j * step;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[j][i] = 0.f;
            load8<W>(o[j], res + c, p.H - c);
        }
        R* dst = static_cast<R*>(p.residual_out) + row * p.ldr;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid * 8 + j * step;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += o[j][i];
            store8<W>(dst + c, v[j], p.H - c);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    ss = row_reduce<false>(ss, sum_buf, warp_row);
    const float inv_rms = rsqrtf(ss / p.H + p.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * inv_rms * g[j][i];
    if (p.out) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.ldo;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid * 8 + j * step;
            store8<W>(out + c, v[j], p.H - c);
        }
    }
    if (!p.q) return;
    float amax[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        amax[j] = 0.f;
        // (elements past the row's end may be 0 * infinity)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (tid * 8 + j * step + i < p.H) amax[j] = max_nan(amax[j], fabsf(v[j][i]));
    }
    float* scale = p.q_scale + row * p.n_groups;
    uint8_t* q = p.q + row * p.H;
    if (p.group == p.H) {
        float m = amax[0];
#pragma unroll
        for (int j = 1; j < VPT; ++j) m = max_nan(m, amax[j]);
        const Scale of(row_reduce<true>(m, max_buf, warp_row));
        if (tid == 0) scale[0] = of.s;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid * 8 + j * step;
            store8_e4m3<W>(q + c, v[j], of, p.H - c);
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j) store_group<W>(p, tid * 8 + j * step, v[j], amax[j], scale, q);
    }
}

// Rows of any length that start at the same distance from a 16-byte boundary in
// every tensor (contiguous ones do): a thread's eight elements are an aligned
// piece, `s` elements before a multiple of eight columns, and only the row's
// first and last piece go by single elements.  The weights, whose distance
// differs, come as two pieces that are shifted together.  A scale group ends
// inside a piece, always after s elements: the maxima of both sides, and the
// scales, cross to the neighbouring thread.  A row to a warp (WARP) or a CTA,
// one piece to a thread as far as a CTA goes: with four the straight code of a row
// (64 KB) ran as fast as its instructions came from L2 (16384 x 777: 2.7 times the
// time with one).  What bounds it: the barriers and the dependent loads of a row, two
// or three rows an SM in flight (16384 x 5001, 242 us, 3.1 TB/s).
__device__ __forceinline__ uint4 shift_eight(const uint4& a, const uint4& b, int s)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (s & 4) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (s & 2) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (s & 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The elements [first, last) of a piece; the others stay as they are.
template <class T>
__device__ __forceinline__ void load_piece(float (&v)[8], const T* p, int first, int last)
{
    if (first == 0 && last == 8) {
        load8<8>(v, p, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= first && i < last) v[i] = static_cast<float>(p[i]);
    }
}

template <class T>
__device__ __forceinline__ void store_piece(T* p, const float (&v)[8], int first, int last)
{
    if (first == 0 && last == 8) {
        store8<8>(p, v, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= first && i < last) p[i] = static_cast<T>(v[i]);
    }
}

template <int VPT, int RES, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpRows * 32 : kOffsetThreads) norm_offset_kernel(const NormParams p)
{
    constexpr int kGroups = WARP ? kWarpRowMax / 32 : kOffsetThreads * VPT * 8 / 32;
    using R = typename std::conditional<RES == 2, float, __nv_bfloat16>::type;
    __shared__ float sum_buf[32], max_buf[32], edge[VPT][33];
    __shared__ float2 of_groups[WARP ? kWarpRows : 1][kGroups];    // Scale of each
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = WARP ? static_cast<long long>(blockIdx.x) * kWarpRows + warp : blockIdx.x;
    const int threads = WARP ? 32 : blockDim.x, tid = WARP ? lane : threadIdx.x;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (row >= p.T) return;     // whole warps only
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + row * p.ldx;
    const __nv_bfloat16* weight = static_cast<const __nv_bfloat16*>(p.weight);
    const int s = static_cast<int>(reinterpret_cast<uintptr_t>(x) >> 1) & 7;
    float v[VPT][8], g[VPT][8];
    int lo[VPT], first[VPT], last[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        lo[j] = (tid + j * threads) * 8 - s;
        first[j] = max(0, -lo[j]);
        last[j] = min(8, p.H - lo[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = g[j][i] = 0.f;
        load_piece(v[j], x + lo[j], first[j], last[j]);
        const int c = lo[j] + s;
        if (s == 0) {
            load_piece(g[j], weight + lo[j], first[j], last[j]);
        } else if (c < 8 || c + 8 > p.H) {       // (no aligned piece of the weights, even if it is one of the row's)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= first[j] && i < last[j]) g[j][i] = __bfloat162float(weight[lo[j] + i]);
        } else {
            const uint4* w = reinterpret_cast<const uint4*>(weight + c);
            const uint4 u = shift_eight(__ldg(w - 1), __ldg(w), 8 - s);
            unpack8(g[j], u);
        }
    }
    if constexpr (RES != 0) {
        const R* res = static_cast<const R*>(p.residual) + row * p.ldr;
        R* dst = static_cast<R*>(p.residual_out) + row * p.ldr;
        float o[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[j][i] = 0.f;
            load_piece(o[j], res + lo[j], first[j], last[j]);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += o[j][i];
            store_piece(dst + lo[j], v[j], first[j], last[j]);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    ss = row_reduce<false>(ss, sum_buf, WARP);
    const float inv_rms = rsqrtf(ss / p.H + p.eps);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.ldo;
    float before[VPT], after[VPT];      // largest magnitudes of the elements before and from s on
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        before[j] = after[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[j][i] = v[j][i] * inv_rms * g[j][i];
            const float a = i >= first[j] && i < last[j] ? fabsf(v[j][i]) : 0.f;    // (0 * infinity past the ends)
            if (i < s) before[j] = max_nan(before[j], a);
            else after[j] = max_nan(after[j], a);
        }
        if (p.out) store_piece(out + lo[j], v[j], first[j], last[j]);
    }
    if (!p.q) return;
    float* scale = p.q_scale + row * p.n_groups;
    uint8_t* q = p.q + row * p.H;
    float2* own = of_groups[WARP ? warp : 0];
    int shift = 31;                     // of a column to its group
    if (p.group == p.H) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) m = max_nan(m, max_nan(before[j], after[j]));
        const Scale of(row_reduce<true>(m, max_buf, WARP));
        if (tid == 0) {
            scale[0] = of.s;
            own[0] = make_float2(of.s, of.inverse);
        }
    } else {
        shift = 31 - __clz(p.group);
        if (!WARP) {
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) edge[j][warp] = before[j];
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float next = __shfl_down_sync(0xffffffffu, before[j], 1);
            if (WARP) {
                const float over = j + 1 < VPT ? __shfl_sync(0xffffffffu, before[j + 1 < VPT ? j + 1 : 0], 0) : 0.f;
                if (lane == 31) next = over;
            } else if (lane == 31) {
                next = warp + 1 < threads / 32 ? edge[j][warp + 1] : j + 1 < VPT ? edge[j + 1 < VPT ? j + 1 : 0][0] : 0.f;
            }
            float m = max_nan(after[j], next);
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
            if (p.group > 32) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 4));
            if (p.group > 64) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
            const int c = lo[j] + s;
            if ((c & (p.group - 1)) == 0 && c < p.H) {
                const Scale of(m);
                scale[c >> shift] = of.s;
                own[c >> shift] = make_float2(of.s, of.inverse);
            }
        }
    }
    if (WARP) __syncwarp();
    else __syncthreads();
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (last[j] <= 0) continue;
        const int c = lo[j] + s;
        const Scale s0(own[max(c - 8, 0) >> shift]), s1(own[min(c, p.H - 1) >> shift]);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = e4m3x2((2 * i < s ? s0 : s1).divide(v[j][2 * i]), (2 * i + 1 < s ? s0 : s1).divide(v[j][2 * i + 1]));
        if (first[j] == 0 && last[j] == 8) {
            *reinterpret_cast<uint2*>(q + lo[j]) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= first[j] && i < last[j]) q[lo[j] + i] = static_cast<uint8_t>(h[i / 2] >> (8 * (i & 1)));
        }
    }
}

// f(residual kind)
template <class F>
cudaError_t by_residual(const NormParams& p, F f)
{
    if (!p.residual) return f(std::integral_constant<int, 0>());
    if (!p.residual_f32) return f(std::integral_constant<int, 1>());
    return f(std::integral_constant<int, 2>());
}

template <int VPT, bool WARP>
cudaError_t launch_rows(const NormParams& p, cudaLaunchConfig_t lc, int num_sms)
{
    return by_residual(p, [&](auto res) {
        const auto kernel = norm_rows_kernel<VPT, decltype(res)::value, WARP>;
        // about as many CTAs as the SMs hold at once (64, 128 and up to 176 registers a thread)
        const int threads = static_cast<int>(lc.blockDim.x);
        const int per_sm = WARP ? (VPT == 1 ? 3 : VPT == 2 ? 2 : 1) : (VPT <= 2 ? 1024 : 512) / threads;
        const int most = num_sms * per_sm, rows = WARP ? kWarpRows : 1;
        const int want = (p.T - 1) / rows + 1;
        lc.gridDim = dim3(want < most ? want : most);
        return cudaLaunchKernelEx(&lc, kernel, p);
    });
}

template <int W, int VPT>
cudaError_t launch_any(const NormParams& p, const cudaLaunchConfig_t& lc, int warp_row)
{
    return by_residual(p, [&](auto res) { return cudaLaunchKernelEx(&lc, norm_kernel<W, VPT, decltype(res)::value>, p, warp_row); });
}

template <int W>
cudaError_t launch_any(const NormParams& p, const cudaLaunchConfig_t& lc, int warp_row, int vpt)
{
    if (vpt <= 1) return launch_any<W, 1>(p, lc, warp_row);
    if (vpt <= 2) return launch_any<W, 2>(p, lc, warp_row);
    return launch_any<W, 4>(p, lc, warp_row);
}

int up32(int n) { return (n + 31) / 32 * 32; }

template <int VPT, bool WARP>
cudaError_t launch_offset(const NormParams& p, cudaLaunchConfig_t lc, int pieces)
{
    lc.gridDim = dim3(WARP ? (p.T - 1) / kWarpRows + 1 : p.T);
    lc.blockDim = dim3(WARP ? kWarpRows * 32 : up32((pieces + VPT - 1) / VPT));
    return by_residual(p, [&](auto res) { return cudaLaunchKernelEx(&lc, norm_offset_kernel<VPT, decltype(res)::value, WARP>, p); });
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int width, bool same_offset, int num_sms, cudaStream_t stream, bool pdl)
{
    const int vecs = (p.H + 7) / 8;
    const int warp_row = p.H <= kWarpRowMax;
    cudaLaunchConfig_t lc = {};
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = pdl ? 1 : 0;
    if (width == 8) {
        if (warp_row) {
            lc.blockDim = dim3(kWarpRows * 32);
            if (vecs <= 32) return launch_rows<1, true>(p, lc, num_sms);
            if (vecs <= 64) return launch_rows<2, true>(p, lc, num_sms);
            return launch_rows<4, true>(p, lc, num_sms);
        }
        if (vecs <= 2048) {
            const int vpt = vecs <= 1024 ? 2 : 4;
            lc.blockDim = dim3(up32((vecs + vpt - 1) / vpt));
            return vpt == 2 ? launch_rows<2, false>(p, lc, num_sms) : launch_rows<4, false>(p, lc, num_sms);
        }
        // longer rows fill the registers without a second row in flight
        lc.gridDim = dim3(p.T);
        lc.blockDim = dim3(up32((vecs + 3) / 4));
        return launch_any<8>(p, lc, 0, 4);
    }
    // Pieces, where the rows allow them, against pairs: 16384 x 1002 47 us and 103,
    // 16384 x 2002 92 and 87, 16384 x 2934 149 and 133 (fewer barriers); against
    // single elements: 16384 x 777 45 and 97, 16384 x 5001 242 and 509.  (Up to
    // seven elements of a row's first piece are not the row's.)
    const int pieces = (p.H + 14) / 8;
    if (same_offset && pieces <= 2 * kOffsetThreads && (width == 1 || warp_row)) {
        if (pieces <= 32) return launch_offset<1, true>(p, lc, pieces);
        if (pieces <= kOffsetThreads) return launch_offset<1, false>(p, lc, pieces);
        return launch_offset<2, false>(p, lc, pieces);
    }
    int vpt = warp_row ? (vecs + 31) / 32 : (vecs + 1023) / 1024;
    if (vpt == 3) vpt = 4;
    lc.gridDim = dim3(warp_row ? (p.T - 1) / kWarpRows + 1 : p.T);
    lc.blockDim = dim3(warp_row ? kWarpRows * 32 : up32((vecs + vpt - 1) / vpt));
    return width == 2 ? launch_any<2>(p, lc, warp_row, vpt) : launch_any<1>(p, lc, warp_row, vpt);
}

}  // namespace tovl
