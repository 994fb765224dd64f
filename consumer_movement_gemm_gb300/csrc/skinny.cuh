// skinny.cuh -- products of a few rows with a streamed weight matrix: the
// parts that the expert layer for few tokens and the 4-bit products share.
//
// out[r][n] = sum_k x[r][k] W[k][n] with at most 64 rows is bound by reading
// W once, so W is laid in shared memory by TMA and everything else fits
// around that stream.  A CTA owns a contiguous range of 4 KB weight blocks
// (64 columns x 32 rows of bf16, or 64 columns x 128 rows of 4 bits) in the
// order (tile of 64 columns, k); its 8 warps take the blocks in turn.  Every
// warp has its own ring of stages, filled by its own lane 0, so no warp waits
// for another one inside a tile, and the ring runs on across tiles (and
// across the two products of an expert layer: weights depend on nothing).
// The sum over a tile's blocks ends in a cross-warp reduction in shared
// memory; tiles that the even split cuts are finished by the last CTA to
// arrive, which adds the parts in the order of k (same bits every time).
//
// The matrix instruction is the warp-level m16n8k16 with the weights as the
// 16-row operand: at most 8 rows cost one instruction per 16 columns x 16
// rows of W, registers feed it directly (4-bit weights never go back to
// shared memory), and even 64 rows need less of the tensor pipe than the
// stream leaves time for.
#pragma once
#include <cuda_bf16.h>
#include "common.cuh"
#include "ops.cuh"
#include "sync.cuh"

namespace tovl {
namespace skinny {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = 64;                         // columns of a tile
constexpr int kBlockBytes = 4096;                 // weight bytes of a block
constexpr int kRowsBf16 = 32;                     // rows of W in a block, bf16
constexpr int kRowsQ4 = 128;                      // rows of W in a block, 4 bits
constexpr int kStagesBf16 = 5;                    // 160 KB in flight per SM
constexpr int kStagesQ4 = 4;                      // 128 KB + scales
constexpr int kScaleBytes = 512;                  // scales of a block (group >= 32)
constexpr int kZeroBytes = 256;
constexpr int kMetaBytes = kScaleBytes + kZeroBytes;
constexpr int kRedPitch = kCols + 4;              // 8 x 4 lanes of an accumulator store hit 32 banks
constexpr int kRedFloats = kWarps * 8 * kRedPitch;

constexpr int stages(bool q4) { return q4 ? kStagesQ4 : kStagesBf16; }
constexpr int block_rows(bool q4) { return q4 ? kRowsQ4 : kRowsBf16; }
// ring (1 KB aligned), block scales, cross-warp reduction, barriers
constexpr int ring_bytes(bool q4) { return kWarps * stages(q4) * kBlockBytes; }
constexpr int meta_bytes(bool q4) { return q4 ? kWarps * stages(q4) * kMetaBytes : 0; }
constexpr int base_smem(bool q4)
{
    return 1024 + ring_bytes(q4) + meta_bytes(q4) + kRedFloats * 4 + kWarps * stages(q4) * 8;
}

// ------------------------------------------------------------ instructions
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint2 ld_shared_u2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_shared_u1(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// d += a x b: a 16 x 16 (rows: weight columns), b 16 x 8 (columns: tokens)
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 d = __hsub2(reinterpret_cast<const __nv_bfloat162&>(a), reinterpret_cast<const __nv_bfloat162&>(b));
    return reinterpret_cast<const uint32_t&>(d);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Four e4m3 values as two bf16 pairs (exact: 4 significant bits, exponents
// from -9 to 8).
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t v)
{
    uint32_t h0, h1;
    asm("{.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(h0), "=r"(h1)
        : "r"(v));
    const float2 a = __half22float2(reinterpret_cast<const __half2&>(h0));
    const float2 b = __half22float2(reinterpret_cast<const __half2&>(h1));
    return make_uint2(ptx::pack_bf16x2(a.x, a.y), ptx::pack_bf16x2(b.x, b.y));
}

// ------------------------------------------------------------ the warp's ring
// Stage s of a warp: 4 KB of weights (1 KB aligned, 128-byte swizzle), for
// 4-bit weights also the block's scales and zeros, and one mbarrier.
template <bool Q4>
struct Ring {
    static constexpr int S = stages(Q4);
    uint8_t* w;          // this warp's stages
    uint8_t* meta;
    uint64_t* full;
    int fill = 0;        // next stage to fill
    int take = 0;        // next stage to read
    uint32_t parity = 0;

    __device__ void init(uint8_t* smem, int warp)
    {
        w = smem + warp * S * kBlockBytes;
        meta = smem + ring_bytes(Q4) + warp * S * kMetaBytes;
        full = reinterpret_cast<uint64_t*>(smem + ring_bytes(Q4) + meta_bytes(Q4) + kRedFloats * 4) + warp * S;
    }

    __device__ void init_barriers()
    {
        for (int s = 0; s < S; ++s) ptx::mbar_init(full + s, 1);
    }

    // One lane: fetch block (column n, weight row k, expert e).  `group`:
    // rows of W per scale (4-bit weights).
    __device__ void issue(const WeightMaps& m, int n, int k, int e, int group, bool has_zero, uint64_t pol)
    {
        uint8_t* dst = w + fill * kBlockBytes;
        uint64_t* bar = full + fill;
        if constexpr (Q4) {
            const int groups = kRowsQ4 / group;
            const uint32_t sb = groups * kCols * 2, zb = has_zero ? groups * kCols : 0;
            ptx::mbar_arrive_expect_tx(bar, kBlockBytes + sb + zb);
            ptx::tma_load_3d_hint(dst, &m.w, bar, n, k / 8, e, pol);
            ptx::tma_load_3d_hint(dst + kBlockBytes / 2, &m.w, bar, n + kCols / 2, k / 8, e, pol);
            uint8_t* md = meta + fill * kMetaBytes;
            ptx::tma_load_3d_hint(md, &m.scale, bar, n, k / group, e, pol);
            if (has_zero) ptx::tma_load_3d_hint(md + kScaleBytes, &m.zero, bar, n, k / group, e, pol);
        } else {
            ptx::mbar_arrive_expect_tx(bar, kBlockBytes);
            ptx::tma_load_3d_hint(dst, &m.w, bar, n, k, e, pol);
        }
    }
    __device__ void filled() { fill = fill + 1 == S ? 0 : fill + 1; }

    __device__ void wait(const Ctrl& ctrl, long long timeout_ns) { mbar_wait(full + take, parity, ctrl, timeout_ns); }
    __device__ uint32_t stage() const { return ptx::smem_u32(w + take * kBlockBytes); }
    __device__ uint32_t stage_meta() const { return ptx::smem_u32(meta + take * kMetaBytes); }
    __device__ void taken()
    {
        if (++take == S) {
            take = 0;
            parity ^= 1;
        }
    }
};

// ------------------------------------------------------------ the rows' fragments
// The k16 step's operand b gives lane 4g + t the rows' columns 2t, 2t+1 and
// 2t+8, 2t+9 of token g.  The order of k is free as long as both operands use
// the same, so a lane loads 16 bytes (8 consecutive k, an octet) of its token
// and both k16 steps of 32 rows of W come from them.
//
// bf16 weights: ldmatrix reads 8 rows of W per matrix, and the 128-byte
// swizzle keeps them apart in the banks only if their indexes differ modulo
// 8.  Lane t therefore uses pair (t ^ i) of its octet in quarter-step i
// (rows 8t + 2(t^i) + {0,1}: all different modulo 8), which needs this swap of
// the loaded pairs.
__device__ __forceinline__ uint4 rotate_pairs(uint4 v, int t)
{
    if (t & 1) v = make_uint4(v.y, v.x, v.w, v.z);
    if (t & 2) v = make_uint4(v.z, v.w, v.x, v.y);
    return v;
}

// acc[mt][nt]: 16 columns x 8 rows.  One block of 32 x 64 bf16 weights.
template <int NT, bool LO>
__device__ __forceinline__ void block_bf16(float (&acc)[4][NT][4], const uint4 (&b)[NT], const uint4 (&bl)[NT],
                                           uint32_t stage, int lane)
{
    const int m = lane >> 3, r = lane & 7;
    const int tp = r >> 1;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int low = 2 * (tp ^ (2 * s + (m >> 1))) + (r & 1);   // row of W modulo 8
        const uint32_t row = stage + (8 * tp + low) * 128;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            uint32_t a[4];
            ldmatrix_x4_trans(a, row + (((2 * mt + (m & 1)) ^ low) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma(acc[mt][nt], a[0], a[1], a[2], a[3], s ? b[nt].z : b[nt].x, s ? b[nt].w : b[nt].y);
                if (LO) mma(acc[mt][nt], a[0], a[1], a[2], a[3], s ? bl[nt].z : bl[nt].x, s ? bl[nt].w : bl[nt].y);
            }
        }
    }
}

// Column of accumulator row g (and g + 8) of m-tile mt.
template <bool Q4>
__device__ __forceinline__ int acc_col(int mt, int g, int upper)
{
    // 4-bit: lane group g owns four neighbouring columns of each half tile;
    // the order 0 4 1 5 2 6 3 7 of the groups keeps the 16-byte reads of a
    // quarter warp in different banks
    if (Q4) return (mt >> 1) * 32 + 4 * ((g >> 1) | ((g & 1) << 2)) + 2 * (mt & 1) + upper;
    return mt * 16 + g + 8 * upper;
}

// The four bf16 pairs (nibble - zero) of a packed word, rows in order.
// 0x4300 | nibble is the bf16 number 128 + nibble, and 128 + zero is one too,
// so the difference is exact; the scale is applied to the fp32 sum of the
// group, so no weight is rounded.
__device__ __forceinline__ void unpack(uint32_t (&p)[4], uint32_t word, uint32_t zero2)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = sub_bf16x2(((word >> (4 * i)) & 0x000f000fu) | 0x43004300u, zero2);
}

// One block of 128 x 64 4-bit weights.  b[R][nt]: octet t of rows 32R .. 32R+31
// of token g.  sx: the tokens' activation scales (1 for bf16 activations).
template <int NT, bool LO, bool XS>
__device__ __forceinline__ void block_q4(float (&acc)[4][NT][4], const uint4 (&b)[4][NT], const uint4 (&bl)[4][NT],
                                         const float2 (&sx)[NT], uint32_t stage, uint32_t meta, int gsteps, bool has_zero,
                                         int lane)
{
    const int g = lane >> 2, t = lane & 3;
    const int c = (g >> 1) | ((g & 1) << 2);
    float part[4][NT][4];
    uint32_t z[2][4];
    int gi = 0;
#pragma unroll
    for (int R = 0; R < 4; ++R) {
        if ((R & (gsteps - 1)) == 0) {
            gi = R / gsteps;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[mt][nt][i] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t zz = has_zero ? ld_shared_u1(meta + kScaleBytes + gi * kCols + h * 32 + 4 * c) : 0x08080808u;
#pragma unroll
                for (int i = 0; i < 4; ++i) z[h][i] = 0x43004300u + ((zz >> (8 * i)) & 0x7fu) * 0x00010001u;
            }
        }
        const int row = 4 * R + t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 v = ld_shared_u4(stage + h * (kBlockBytes / 2) + row * 128 + ((c ^ (row & 7)) << 4));
            uint32_t p0[4], p1[4], p2[4], p3[4];
            unpack(p0, v.x, z[h][0]);
            unpack(p1, v.y, z[h][1]);
            unpack(p2, v.z, z[h][2]);
            unpack(p3, v.w, z[h][3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 x = b[R][nt];
                mma(part[2 * h][nt], p0[0], p1[0], p0[1], p1[1], x.x, x.y);
                mma(part[2 * h + 1][nt], p2[0], p3[0], p2[1], p3[1], x.x, x.y);
                mma(part[2 * h][nt], p0[2], p1[2], p0[3], p1[3], x.z, x.w);
                mma(part[2 * h + 1][nt], p2[2], p3[2], p2[3], p3[3], x.z, x.w);
                if (LO) {
                    const uint4 y = bl[R][nt];
                    mma(part[2 * h][nt], p0[0], p1[0], p0[1], p1[1], y.x, y.y);
                    mma(part[2 * h + 1][nt], p2[0], p3[0], p2[1], p3[1], y.x, y.y);
                    mma(part[2 * h][nt], p0[2], p1[2], p0[3], p1[3], y.z, y.w);
                    mma(part[2 * h + 1][nt], p2[2], p3[2], p2[3], p3[3], y.z, y.w);
                }
            }
        }
        if ((R & (gsteps - 1)) == gsteps - 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 s2 = ld_shared_u2(meta + gi * (kCols * 2) + (h * 32 + 4 * c) * 2);
                const float s[4] = {bf16_lo(s2.x), bf16_hi(s2.x), bf16_lo(s2.y), bf16_hi(s2.y)};
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float f = s[2 * u + (i >> 1)];
                            if (XS) f *= (i & 1) ? sx[nt].y : sx[nt].x;
                            acc[2 * h + u][nt][i] = fmaf(f, part[2 * h + u][nt][i], acc[2 * h + u][nt][i]);
                        }
            }
        }
    }
}

// ------------------------------------------------------------ cross-warp sums
// Writes n-tile nt of the warp's accumulators to red[warp][row][column].
template <bool Q4, int NT>
__device__ __forceinline__ void store_red(float* red, const float (&acc)[4][NT][4], int nt, int warp, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    float* r = red + (warp * 8 + 2 * t) * kRedPitch;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) r[(i & 1) * kRedPitch + acc_col<Q4>(mt, g, i >> 1)] = acc[mt][nt][i];
}

// Whole CTA: counts this CTA's arrival on a tile that n CTAs share; true (for
// every thread) in the last one, whose reads of the others' parts are then
// ordered after their writes.  The last arrival leaves the counter at zero.
__device__ __forceinline__ bool last_arrival(int* counter, int n, int* flag)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const bool last = ptx::atom_add_acq_rel_gpu(counter, 1) == n - 1;
        if (last) ptx::st_relaxed_gpu(counter, 0);
        *flag = last;
        __threadfence();
    }
    __syncthreads();
    return *flag != 0;
}

// The even split of `total` blocks: CTA c owns [c * per, (c + 1) * per).
// At least one block per warp, so that a small product is not cut finer than
// its CTAs can use.
__device__ __forceinline__ int blocks_per_cta(int total, int grid)
{
    int per = (total + grid - 1) / grid;
    if (per < kWarps) per = kWarps;
    return (per + 1) & ~1;     // even: gate and up blocks stay with the same warps
}

}  // namespace skinny
}  // namespace tovl
