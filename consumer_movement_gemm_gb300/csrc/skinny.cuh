// skinny.cuh -- products of a few rows with a streamed weight matrix: the
// engine that the expert layer for few tokens and the 4-bit products share.
//
// out[r][n] = sum_k x[r][k] W[k][n] with at most 64 rows is bound by reading
// W once, so W is laid in shared memory by TMA and everything else fits
// around that stream.
//
// Units.  A unit is 512 columns x 32 rows of bf16 (32 KB) or x 256 rows of 4
// bits (64 KB).  Its columns are dealt to the CTA's warps (8 of 64 columns for
// bf16; 16 of 32 for 4-bit weights, whose unpacking needs twice the warps to
// hide its latencies), a 4 KB block each, so neighbouring warps read neighbouring
// pieces of the same rows at the same time: measured on GB300, a stream of such
// 1 KB wide rows reaches 6.67 TB/s, the same boxes with the warps along k (each
// 128-byte piece alone) 5.85.  A warp owns its columns, so nothing is summed
// across warps and no warp waits for another one; each has its own ring of
// stages (4 blocks of bf16 weights, 2 of 4-bit weights: 128 KB in flight per SM), filled by
// its own lane 0, that runs on across tiles and across the two products of an
// expert layer (weights depend on nothing).  The few rows of x pass through
// shared memory once per CTA in 16 KB chunks, as bf16 or (4-bit weights) turned
// into fp16, where all warps read them.
//
// Items.  The units of a product, in the order (matrix, tile of 512 columns,
// k), are cut into items.  With little work there is one item per CTA; from 3 MB
// of weights per CTA on, one of three quarters of an even share and then small
// ones, an eighth of it, by ticket, because the SMs do not get the same share of
// the memory (an even static deal of 2.3 GB ended between 160 and 229 us).  An
// item writes the fp32 sums of each tile that it touches to the workspace, under
// the number of its part of the tile; then all CTAs, after a grid barrier (expert
// layer), or the last CTA to finish a part of the tile (product alone) add the
// parts in the order of k.  Which CTA took an item changes nothing: the same bits
// every time.
//
// The matrix instruction is the warp-level m16n8k16 with the weights as the
// 16-row operand: at most 8 rows cost one instruction per 16 columns x 16
// rows of W, registers feed it directly (4-bit weights never go back to
// shared memory), and the tensor pipe has time for 64 rows of bf16.  4-bit
// weights as the tensor-memory operand of tcgen05.mma were built and dropped: two
// barriers and 520 instructions per 2 KB against 400, 16 x 7168 x 32768 57 us
// against 46.
//
// What bounds it.  bf16: memory (13 tokens of an expert layer, 2.3 GB, 6.5 TB/s).
// 4 bits: the instructions that turn a block into operands, about 335 per 2 KB
// with up to 8 rows and 400 with 16, four warps a scheduler to hide their
// latencies (49 % of the issue slots, 36 % of the integer pipe, 32 % of the tensor
// pipe): 2.8 TB/s with 16 rows, 4.0 with one.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "common.cuh"
#include "ops.cuh"
#include "sync.cuh"

namespace tovl {
namespace skinny {

constexpr int kTileCols = 512;
constexpr int kScaleBytes = 512;                  // scales of a 4-bit block (group >= 32)
constexpr int kZeroBytes = 256;
constexpr int kItemsPerCta = 8;                   // small items of an even share, with tickets
constexpr int kTicketBytes = 3 << 20;             // an even share of the weights from which tickets are worth it
constexpr int kMaxItems = kMaxGrid * kItemsPerCta;

// G: rows per scale (0: bf16 weights).
template <int G>
struct Shape {
    static constexpr bool Q4 = G != 0;
    static constexpr int kWarps = Q4 ? 16 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kCols = kTileCols / kWarps;          // columns of a warp
    static constexpr int kRows = Q4 ? 256 : 32;               // rows of W in a block: 4 KB
    static constexpr int kBlockBytes = 4096;
    static constexpr int kUnitBytes = kBlockBytes * kWarps;
    static constexpr int kMetaBytes = Q4 ? kScaleBytes + kZeroBytes : 0;
    static constexpr int kStages = Q4 ? 2 : 4;                // 128 KB in flight per SM
    static constexpr int kMT = kCols / 16;                    // 16-column accumulator tiles
    static constexpr int kRing = kWarps * kStages * (kBlockBytes + kMetaBytes + 8);   // 1 KB aligned
};

// Rows of x wait in shared memory in chunks of units: 16 KB of bf16 for NT * 8
// rows, with their second parts (LO) behind them; three chunks and a barrier
// for each.
constexpr int kChunkBytes = 16384;
constexpr int kScalesOfChunk = 256;               // e4m3: a scale per row and 128 columns
constexpr int kChunkStride = kChunkBytes + kScalesOfChunk * 4;
constexpr int kRowBuffers = 3 * kChunkStride + 32 + 16 * 32;    // also the chunks' barriers and the warps' places

// What the rows of a product are.
enum class Rows {
    kBf16,      // bf16; with 4-bit weights turned into fp16 with a power of two per 128 columns
    kPair,      // bf16 and what its rounding left over, bf16 (bf16 weights only)
    kHalf,      // fp16 with a scale per 128 columns (4-bit weights only)
    kE4m3       // e4m3 with a scale per 128 columns (4-bit weights only)
};
template <int G, int NT, bool LO>
constexpr int chunk_units() { return kChunkBytes / (NT * 8 * (LO ? 2 : 1) * Shape<G>::kRows * 2); }

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

// 16 bytes that are read once
__device__ __forceinline__ uint4 ld_stream(const uint32_t* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Number in another CTA of the cluster, by its shared::cluster address.
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ uint2 ld_shared_u2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_f1(uint32_t addr, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u1(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, "
        "%5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(pol)
        : "memory");
}

// mbarriers by shared address
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait (the CTA's own copies and warps; a bound against logic errors).
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, const Ctrl& ctrl, long long timeout_ns)
{
    if (mbar_try(bar, parity)) return;
    const uint64_t start = ptx::globaltimer();
    for (uint32_t i = 1; !mbar_try(bar, parity); ++i) {
        if ((i & 255) == 0 && ptx::globaltimer() - start > static_cast<uint64_t>(timeout_ns)) {
            record_error(ctrl, kErrTimeout);
            return;
        }
    }
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

// The same in fp16.
__device__ __forceinline__ void mma_h(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a x b
__device__ __forceinline__ void mma_h_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t sub_h2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t fma_h2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// (a & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Four e4m3 values as two fp16 pairs (exact).
__device__ __forceinline__ uint2 e4m3x4_to_half(uint32_t v)
{
    uint2 h;
    asm("{.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(h.x), "=r"(h.y)
        : "r"(v));
    return h;
}

// The power of two that brings numbers of largest exponent field e (bf16, 0
// to 255) below 2^15, and its inverse.  In fp16 so scaled, a bf16 number keeps
// all its bits down to 2^-31 of the largest, and what a smaller one loses is
// 2^-39 of the largest: nothing beside the fp32 sums' own 2^-24.  (The power ends at
// 2^126.  Where the largest is below 2^-112 / scale, the inverse times a weight's
// scale is a subnormal number, and a group's sum loses 2^-124 at most.)
__device__ __forceinline__ float half_scale(uint32_t e) { return __uint_as_float(min(268u - e, 253u) << 23); }
__device__ __forceinline__ float half_unscale(uint32_t e) { return __uint_as_float((254u - min(268u - e, 253u)) << 23); }

// Eight bf16 numbers times f as fp16.
__device__ __forceinline__ uint4 bf16x8_to_half(const uint4& v, float f)
{
    return make_uint4(pack_h2(bf16_lo(v.x) * f, bf16_hi(v.x) * f), pack_h2(bf16_lo(v.y) * f, bf16_hi(v.y) * f),
                      pack_h2(bf16_lo(v.z) * f, bf16_hi(v.z) * f), pack_h2(bf16_lo(v.w) * f, bf16_hi(v.w) * f));
}

// Largest exponent field of eight bf16 numbers.
__device__ __forceinline__ uint32_t max_exponent(const uint4& u)
{
    const uint32_t m = 0x7f807f80u;
    const uint32_t a = max((u.x & m) >> 16, (u.y & m) >> 16), b = max((u.z & m) >> 16, (u.w & m) >> 16);
    const uint32_t c = max(u.x & 0x7f80u, u.y & 0x7f80u), d = max(u.z & 0x7f80u, u.w & 0x7f80u);
    return max(max(a, b), max(c, d)) >> 7;
}

// ------------------------------------------------------------ the warp's ring
// Stage s of a warp: a block of weights (128-byte swizzle), for 4-bit weights
// also its [group][32] scales and zeros, and one mbarrier.  Z: with zeros.
template <int G, bool Z>
struct Ring {
    using P = Shape<G>;
    static constexpr int S = P::kStages;
    uint32_t w, meta, full;    // this warp's stages and barriers (shared addresses)
    int take = 0;              // next stage to read
    uint32_t parity = 0;

    __device__ void init(uint32_t smem, int warp)
    {
        w = smem + warp * S * P::kBlockBytes;
        meta = smem + P::kWarps * S * P::kBlockBytes + warp * S * P::kMetaBytes;
        full = smem + P::kWarps * S * (P::kBlockBytes + P::kMetaBytes) + warp * S * 8;
    }

    __device__ void init_barriers()
    {
        for (int s = 0; s < S; ++s) mbar_init(full + s * 8, 1);
    }

    // One lane: fetch the block at column n, weight row k of matrix e into a stage.
    __device__ __forceinline__ void issue(int fill, const WeightMaps* m, int n, int k, int e, uint64_t pol) const
    {
        const uint32_t dst = w + fill * P::kBlockBytes, bar = full + fill * 8;
        if constexpr (P::Q4) {
            constexpr int kGroups = P::kRows / (G ? G : 1);
            const uint32_t md = meta + fill * P::kMetaBytes;
            mbar_expect(bar, P::kBlockBytes + kGroups * P::kCols * (Z ? 3 : 2));
            tma_load_3d(dst, &m->w, bar, n, k / 8, e, pol);
            tma_load_3d(md, &m->scale, bar, n, k / G, e, pol);
            if (Z) tma_load_3d(md + kScaleBytes, &m->zero, bar, n, k / G, e, pol);
        } else {
            mbar_expect(bar, P::kBlockBytes);
            tma_load_3d(dst, &m->w, bar, n, k, e, pol);
        }
    }
    __device__ __forceinline__ void wait(const Ctrl& ctrl, long long timeout_ns) { bar_wait(full + take * 8, parity, ctrl, timeout_ns); }
    __device__ __forceinline__ uint32_t block() const { return w + take * P::kBlockBytes; }
    __device__ __forceinline__ uint32_t scales() const { return meta + take * P::kMetaBytes; }
    __device__ __forceinline__ void taken()
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
// the same, so a lane reads 16 bytes (8 consecutive k, an octet) of its token
// and both k16 steps of 32 rows of W come from them.  Octet o of row r lies at
// r * pitch + 16 * (o ^ 4 (r & 1)): the two rows that a quarter warp reads
// together use different banks.
struct RowView {
    uint32_t even, odd;      // this lane's octet t of an even (odd) group of 32 k, token g of the first 8
    uint32_t tokens8;        // bytes from one 8 tokens to the next
    uint32_t second;         // bytes to the second parts
    __device__ __forceinline__ uint4 get(int R, int nt, bool lo) const
    {
        return ld_shared_u4(((R & 1) ? odd : even) + (R >> 1) * 128 + nt * tokens8 + (lo ? second : 0));
    }
};

// bf16 weights: ldmatrix reads 8 rows of W per matrix, and the swizzle keeps
// them apart in the banks only if their indexes differ modulo 8.  Lane t
// therefore uses pair (t ^ i) of its octet in quarter-step i (rows 8t +
// 2(t^i) + {0,1}: all different modulo 8), which needs this swap of the
// loaded pairs.
__device__ __forceinline__ uint4 rotate_pairs(uint4 v, int t)
{
    if (t & 1) v = make_uint4(v.y, v.x, v.w, v.z);
    if (t & 2) v = make_uint4(v.z, v.w, v.x, v.y);
    return v;
}

// acc[mt][nt] (16 columns x 8 rows each) += a block of 32 x 64 bf16 weights.
// R: the block's 32 k inside the view.
template <int NT, bool LO>
__device__ __forceinline__ void block_bf16(float (&acc)[4][NT][4], const RowView& x, int R, uint32_t block, int lane)
{
    const int m = lane >> 3, r = lane & 7;
    const int tp = r >> 1;
    uint32_t a[2][4][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int low = 2 * (tp ^ (2 * s + (m >> 1))) + (r & 1);   // row of W modulo 8
        const uint32_t row = block + (8 * tp + low) * 128;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) ldmatrix_x4_trans(a[s][mt], row + (((2 * mt + (m & 1)) ^ low) << 4));
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int l = 0; l < (LO ? 2 : 1); ++l) {
            const uint4 b = rotate_pairs(x.get(R, nt, l), lane & 3);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) mma(acc[mt][nt], a[0][mt][0], a[0][mt][1], a[0][mt][2], a[0][mt][3], b.x, b.y);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) mma(acc[mt][nt], a[1][mt][0], a[1][mt][1], a[1][mt][2], a[1][mt][3], b.z, b.w);
        }
}

// The four fp16 pairs (nibble - zero) of a packed word, rows in order.  fp16
// has room for two nibbles in its fraction: 0x6400 | n is 1024 + n and
// 0x6400 | 16 n is 1024 + 16 n, so one shift serves four pairs; subtracting
// 1024 + zero, or 64 + zero after a sixteenth, is exact.  The scale is applied
// to the fp32 sum of the group: no weight is rounded.
// z0: 1024 + zero, z1: -(64 + zero), in both halves.
__device__ __forceinline__ void unpack(uint32_t (&p)[4], uint32_t word, uint32_t z0, uint32_t z1)
{
    const uint32_t high = word >> 8, sixteenth = 0x2c002c00u;
    p[0] = sub_h2(and_or(word, 0x000f000fu, 0x64006400u), z0);
    p[1] = fma_h2(and_or(word, 0x00f000f0u, 0x64006400u), sixteenth, z1);
    p[2] = sub_h2(and_or(high, 0x000f000fu, 0x64006400u), z0);
    p[3] = fma_h2(and_or(high, 0x00f000f0u, 0x64006400u), sixteenth, z1);
}

// acc[mt][nt] += 128 x 32 4-bit weights in groups of G rows, with zeros (Z) or
// 8 for all.  Lane group g owns the four neighbouring columns 4 c(g), in the
// order c = 0 4 1 5 2 6 3 7 of the groups, and octet rows t, t + 4, ..:
//   words(R)    the four columns' words of octet row 4 R + t
//   zero(q)     their zeros in group q, one a byte (0 .. 15)
//   scale(q)    their scales in group q, bf16
//   x(R, nt)    octet t of rows 32 R .. 32 R + 31 of token g, fp16
// sx: scales of the tokens 2 t and 2 t + 1.
__device__ __forceinline__ int column_group(int g) { return (g >> 1) | ((g & 1) << 2); }

template <int NT, int G, bool Z, class W, class ZF, class SF, class XF>
__device__ __forceinline__ void multiply_q4(float (&acc)[2][NT][4], const float2 (&sx)[NT], W words, ZF zero, SF scale, XF x)
{
    constexpr int kSteps = G / 32;
    float part[2][NT][4];
    uint32_t z0[4], z1[4];
#pragma unroll
    for (int R = 0; R < 4; ++R) {
        const bool first = R % kSteps == 0, last = R % kSteps == kSteps - 1;
        if (first) {
            if constexpr (Z) {
                // the byte of column i under 0x64 (1024 + z), sixteen times it under 0xd4 (-(64 + z))
                const uint32_t zz = zero(R / kSteps) & 0x0f0f0f0fu;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z0[i] = __byte_perm(zz, 0x64u, 0x4040u | i | i << 8);
                    z1[i] = __byte_perm(zz << 4, 0xd4u, 0x4040u | i | i << 8);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z0[i] = 0x64086408u;
                    z1[i] = 0xd480d480u;
                }
            }
        }
        const uint4 v = words(R);
        uint32_t p0[4], p1[4], p2[4], p3[4];
        unpack(p0, v.x, z0[0], z1[0]);
        unpack(p1, v.y, z0[1], z1[1]);
        unpack(p2, v.z, z0[2], z1[2]);
        unpack(p3, v.w, z0[3], z1[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint4 b = x(R, nt);
            if (first) {
                mma_h_first(part[0][nt], p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                mma_h_first(part[1][nt], p2[0], p3[0], p2[1], p3[1], b.x, b.y);
            } else {
                mma_h(part[0][nt], p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                mma_h(part[1][nt], p2[0], p3[0], p2[1], p3[1], b.x, b.y);
            }
            mma_h(part[0][nt], p0[2], p1[2], p0[3], p1[3], b.z, b.w);
            mma_h(part[1][nt], p2[2], p3[2], p2[3], p3[3], b.z, b.w);
        }
        if (last) {
            const uint2 s2 = scale(R / kSteps);
            const float s[4] = {bf16_lo(s2.x), bf16_hi(s2.x), bf16_lo(s2.y), bf16_hi(s2.y)};
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[mt][nt][i] = fmaf(s[2 * mt + (i >> 1)] * ((i & 1) ? sx[nt].y : sx[nt].x), part[mt][nt][i], acc[mt][nt][i]);
        }
    }
}

// The same with the weights of half a ring block: its words (128-byte
// swizzle; the order of the column groups keeps the 16-byte reads of a quarter
// warp in different banks), scales and zeros.
template <int NT, int G, bool Z>
__device__ __forceinline__ void block_q4(float (&acc)[2][NT][4], const RowView& x, const float2 (&sx)[NT],
                                         uint32_t block, uint32_t scales, uint32_t zeros, int lane)
{
    const int t = lane & 3, c = column_group(lane >> 2);
    const uint32_t low = block + t * 128 + ((c ^ t) << 4), high = block + (t + 4) * 128 + ((c ^ (t + 4)) << 4);
    multiply_q4<NT, G, Z>(
        acc, sx, [&](int R) { return ld_shared_u4(((R & 1) ? high : low) + (R >> 1) * 1024); },
        [&](int q) { return ld_shared_u1(zeros + q * 32 + 4 * c); }, [&](int q) { return ld_shared_u2(scales + q * 64 + 8 * c); },
        [&](int R, int nt) { return x.get(R, nt, false); });
}

// ------------------------------------------------------------ items
// One product: matrices x tiles of 512 columns x kb units along k.  Items 0 ..
// grid - 1 are `big` units long, the ones behind them `small`.
struct Product {
    int tiles, kb, total;      // tiles per matrix, units per tile, units
    int big, small, bigs;      // bigs: units of all big items
    int items;
    bool tickets;

    // An item has no fewer units than leave a tile most_parts + 2 parts at most.
    __device__ __forceinline__ void init(int matrices, int N, int K, int rows, int unit_bytes, int grid, int most_parts)
    {
        tiles = (N + kTileCols - 1) / kTileCols;
        kb = (K + rows - 1) / rows;
        total = matrices * tiles * kb;
        const int share = (total + grid - 1) / grid, least = (kb + most_parts - 1) / most_parts;
        tickets = static_cast<long long>(share) * unit_bytes >= kTicketBytes && share > least;
        big = max(tickets ? share - share / 4 : share, max(least, 1));
        small = max((share + kItemsPerCta - 1) / kItemsPerCta, max(least, 1));
        bigs = min(grid * big, total);
        tickets = tickets && bigs < total;
        items = tickets ? grid + (total - bigs + small - 1) / small : (total + big - 1) / big;
    }
    __device__ __forceinline__ int item_of(int unit) const
    {
        return unit < bigs ? unit / big : static_cast<int>(gridDim.x) + (unit - bigs) / small;
    }
    __device__ __forceinline__ int begin(int item) const
    {
        const int grid = gridDim.x;
        return item < grid ? min(item * big, total) : bigs + (item - grid) * small;
    }
    __device__ __forceinline__ int end(int item) const
    {
        const int grid = gridDim.x;
        return min(item < grid ? min((item + 1) * big, bigs) : bigs + (item - grid + 1) * small, total);
    }
    // parts of the tile whose units start at t0
    __device__ __forceinline__ int parts(int t0) const { return item_of(t0 + kb - 1) - item_of(t0) + 1; }
};

// The items that a CTA works on, in order; shared by its warps.  Entry 0 is
// the CTA's own number; warp 0 takes the others by ticket, two ahead of
// where it fetches, and the other warps read them here.  Long enough for one
// CTA to take them all, so that no entry is ever written twice.
struct Queue {
    volatile uint16_t item[kMaxItems + 8];
};
constexpr int kNoItem = 0xffff;

// Item n of this CTA; product.items or more when there is none.
__device__ __forceinline__ int item_at(const Product& pr, const Queue& q, int n, const Ctrl& ctrl, long long timeout_ns)
{
    if (n == 0) return blockIdx.x;
    if (!pr.tickets) return pr.items;
    int v = q.item[n];
    if (v == kNoItem) {
        const uint64_t start = ptx::globaltimer();
        for (int spin = 1; (v = q.item[n]) == kNoItem; ++spin) {
            if ((spin & 255) == 0 && ptx::globaltimer() - start > static_cast<uint64_t>(timeout_ns)) {
                record_error(ctrl, kErrTimeout);
                return pr.items;
            }
        }
    }
    return v;
}

// Whole CTA: waits until all CTAs of the grid have arrived `round` times on
// the counter; what any of them wrote before is visible after.  Bounded; the
// counter is cleared by the last CTA of the launch to leave.
__device__ __forceinline__ void grid_barrier(int* counter, int target, const Ctrl& ctrl, long long timeout_ns)
{
    __syncthreads();       // (what the CTA wrote before it is released with thread 0's arrival)
    if (threadIdx.x == 0) {
        ptx::red_add_release_gpu(counter, 1);
        if (ptx::ld_acquire_gpu(counter) < target) {
            const uint64_t start = ptx::globaltimer();
            for (int spin = 1; ptx::ld_acquire_gpu(counter) < target; ++spin) {
                if ((spin & 63) == 0 && ptx::globaltimer() - start > static_cast<uint64_t>(timeout_ns)) {
                    record_error(ctrl, kErrTimeout);
                    break;
                }
            }
        }
    }
    __syncthreads();
}

// The calling thread's number when neighbouring warps of the numbering lie in
// different CTAs: little work is spread over all SMs.
__device__ __forceinline__ int spread_thread()
{
    return ((threadIdx.x >> 5) * gridDim.x + blockIdx.x) * 32 + (threadIdx.x & 31);
}

// Adds the parts of M sums of four neighbouring columns: sum m has n[m] parts,
// `stride` floats apart from part[m] on.  Eight parts of every sum are in
// flight together: the sums are short and the latency is long.
template <int M>
__device__ __forceinline__ void add_parts(float4 (&s)[M], const float* const (&part)[M], const int (&n)[M], long long stride)
{
    int most = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        s[m] = make_float4(0.f, 0.f, 0.f, 0.f);
        most = max(most, n[m]);
    }
    for (int i = 0; i < most; i += 8) {
        float4 v[M][8];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i + u < n[m]) v[m][u] = __ldcg(reinterpret_cast<const float4*>(part[m] + (i + u) * stride));
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i + u < n[m]) s[m].x += v[m][u].x, s[m].y += v[m][u].y, s[m].z += v[m][u].z, s[m].w += v[m][u].w;
    }
}

// The next block that a warp fetches: product, next item of the CTA's list,
// units left of the current one, place of the next.
struct Place {
    int ph, n, left, k, col, matrix, k_end, col_end;
};
static_assert(sizeof(Place) == 32, "16 places behind the row buffers");

// The engine of one warp.  `Calls` provides, for product `ph` (0 or 1):
//   maps(ph), expert(ph, matrix)     where a matrix' weights are
template <int G, bool Z, class Calls>
struct Engine {
    using P = Shape<G>;
    static constexpr bool Q4 = P::Q4;
    const Calls& c;
    const Product* pr;         // the call's products, in shared memory
    Queue* queue;
    int* tickets;              // global counters, one per product
    const Ctrl& ctrl;
    long long timeout_ns;
    int n_products;
    int warp, lane;
    Ring<G, Z> ring;
    uint32_t place;            // this warp's Place (shared address)
    uint32_t rows_buf;         // kRowBuffers bytes (shared address): chunks of rows
    uint32_t chunk_bars;       // their barriers
    uint32_t buf_now = 0, buf_parity = 0;

    // Lane 0: goes on to the next item, of this product or the next one;
    // false where there is none.
    __device__ __forceinline__ bool advance(Place& f) const
    {
        for (; f.ph < n_products; ++f.ph, f.n = 0) {
            const Product& q = pr[f.ph];
            const int n = f.n, id = item_at(q, queue[f.ph], n, ctrl, timeout_ns);
            if (id >= q.items) continue;
            ++f.n;
            if (q.tickets && warp == 0) {
                const int grid = gridDim.x;
                int* counter = tickets + f.ph * kSyncStep;
                if (n == 0) queue[f.ph].item[1] = static_cast<uint16_t>(min(atomicAdd(counter, 1) + grid, q.items));
                queue[f.ph].item[n + 2] = static_cast<uint16_t>(min(atomicAdd(counter, 1) + grid, q.items));
            }
            const int b = q.begin(id), at = b / q.kb;
            f.left = q.end(id) - b;
            f.k = (b - at * q.kb) * P::kRows;
            f.matrix = at / q.tiles;
            f.col = (at - f.matrix * q.tiles) * kTileCols;
            f.k_end = q.kb * P::kRows;
            f.col_end = q.tiles * kTileCols;
            return true;
        }
        return false;
    }

    // Fetches the warp's next block, if there is one (lane 0; the place lives
    // in shared memory, the registers belong to the sums).
    __device__ __forceinline__ void fetch(int stage)
    {
        if (lane != 0) return;
        Place& f = *reinterpret_cast<Place*>(__cvta_shared_to_generic(place));
        if (f.left == 0 && !advance(f)) return;
        const int k = f.k, col = f.col, matrix = f.matrix, ph = f.ph;
        --f.left;
        f.k = k + P::kRows;
        if (k + P::kRows == f.k_end) {
            f.k = 0;
            f.col = col + kTileCols;
            if (col + kTileCols == f.col_end) {
                f.col = 0;
                f.matrix = matrix + 1;
            }
        }
        // weights are read once: they leave the L2 to the parts and the rows
        ring.issue(stage, c.maps(ph), col + warp * P::kCols, k, c.expert(ph, matrix), ptx::l2_policy(1));
    }

    // Before the first barrier of the CTA.
    __device__ __forceinline__ void init(uint8_t* smem, uint8_t* rows)
    {
        rows_buf = ptx::smem_u32(rows);
        chunk_bars = rows_buf + 3 * kChunkStride;
        place = chunk_bars + 32 + warp * static_cast<int>(sizeof(Place));
        ring.init(ptx::smem_u32(smem), warp);
        if (lane == 0) {
            ring.init_barriers();
            if (warp == 0)
                for (int b = 0; b < 3; ++b) mbar_init(chunk_bars + b * 8, P::kWarps);
            Place& f = *reinterpret_cast<Place*>(__cvta_shared_to_generic(place));
            f.ph = f.n = f.left = 0;
            ptx::fence_mbar_init();
        }
    }

    __device__ __forceinline__ void start()
    {
#pragma unroll 1
        for (int s = 0; s < P::kStages; ++s) fetch(s);
    }

    // Whole CTA.  Sums over k units [i0, i1) of a tile for `rows` <= NT * 8
    // rows, written to part[row][n], rows `ld` floats apart (n0: the tile's
    // first column, N: the matrix').  octet(r, k, lo) gives 8 elements of row
    // r from column k on (k < K) as they lie in memory, of the second parts if
    // lo; scale(r, k) the row's scale there.  The rows go through shared
    // memory in chunks, once per CTA; the next chunk is in registers while one
    // is multiplied.
    template <int NT, Rows X, class F, class S>
    __device__ __forceinline__ void segment(int i0, int i1, float* part, long long ld, int rows, int n0, int N, int K, F octet,
                                            S scale)
    {
        constexpr bool LO = X == Rows::kPair;
        constexpr bool kGiven = X == Rows::kHalf || X == Rows::kE4m3;  // scales come with the rows
        constexpr int kUnits = chunk_units<G, NT, LO>();
        static_assert(kUnits >= 1, "rows of one unit fit a chunk");
        constexpr int kOctets = kUnits * P::kRows / 8;                 // of a row in a chunk
        constexpr int kPitch = kOctets * 16;
        constexpr int kPer = kChunkBytes / 16 / P::kThreads;           // octets of a thread
        constexpr int kScales = Q4 ? kUnits * P::kRows / kXScaleGroup : 1;   // of a row in a chunk
        float acc[P::kMT][NT][4];
#pragma unroll
        for (int mt = 0; mt < P::kMT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[mt][nt][j] = 0.f;
        const int g = lane >> 2, t = lane & 3;
        const int tid = warp * 32 + lane;
        uint4 next[kPer];
        float next_scale = 0.f;
        // this thread's octets of the chunk that starts at unit u
        const auto get = [&](int u) {
            const int k0 = u * P::kRows, k1 = min(K, i1 * P::kRows);
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                const int at = tid + x * P::kThreads, r = at / kOctets, k = k0 + (at % kOctets) * 8;
                const int row = LO ? r % (NT * 8) : r;
                next[x] = make_uint4(0, 0, 0, 0);     // (rows of W past the last one are zeros; so must these be)
                if (row < rows && k < k1) next[x] = octet(row, k, LO && r >= NT * 8);
            }
            if (kGiven && tid < kScales * NT * 8) {
                const int r = tid / kScales, k = k0 + tid % kScales * kXScaleGroup;
                next_scale = r < rows && k < k1 ? scale(r, k) : 0.f;
            }
        };
        // writes them to buffer c and counts this warp's arrival there
        const auto put = [&](uint32_t c) {
            const uint32_t buf = rows_buf + c * kChunkStride;
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                const int at = tid + x * P::kThreads, r = at / kOctets, o = at % kOctets;
                uint4 v = next[x];
                if constexpr (X == Rows::kE4m3) {
                    const uint2 a = e4m3x4_to_half(v.x), b = e4m3x4_to_half(v.y);
                    v = make_uint4(a.x, a.y, b.x, b.y);
                }
                if constexpr (Q4 && X == Rows::kBf16) {
                    // 16 neighbouring lanes hold the 128 columns
                    uint32_t e = max_exponent(v);
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, d));
                    const float f = half_scale(e);
                    v = bf16x8_to_half(v, f);
                    if ((lane & 15) == 0) st_shared_f1(buf + kChunkBytes + (r * kScales + o / 16) * 4, half_unscale(e));
                }
                ptx::st_shared_v4(buf + r * kPitch + ((o ^ ((r & 1) << 2)) << 4), v.x, v.y, v.z, v.w);
            }
            if (kGiven && tid < kScales * NT * 8) st_shared_f1(buf + kChunkBytes + tid * 4, next_scale);
            __syncwarp();
            if (lane == 0) mbar_arrive(chunk_bars + c * 8);
        };
        // Three buffers in turn.  Chunk c + 1 is written when chunk c begins,
        // into the buffer of chunk c - 2: every warp has arrived at chunk c
        // (the writer has just waited for that), which it does not before it
        // has begun c - 1 and so finished c - 2.  (A segment's first chunk is
        // written when the last one of the segment before it is finished, later
        // still.)  A warp may run a whole chunk ahead of another.
        get(i0);
        put(buf_now);
        if (i0 + kUnits < i1) get(i0 + kUnits);
        for (int u = i0; u < i1; u += kUnits) {
            bar_wait(chunk_bars + buf_now * 8, buf_parity, ctrl, timeout_ns);
            const uint32_t buf = rows_buf + buf_now * kChunkStride;
            if (++buf_now == 3) {
                buf_now = 0;
                buf_parity ^= 1;
            }
            if (u + kUnits < i1) {
                put(buf_now);
                if (u + 2 * kUnits < i1) get(u + 2 * kUnits);
            }
            const uint32_t base = buf + g * kPitch;
            RowView x;
            x.tokens8 = 8 * kPitch;
            x.second = NT * 8 * kPitch;
            const int end = min(kUnits, i1 - u);
#pragma unroll 1
            for (int v = 0; v < end; ++v) {
                ring.wait(ctrl, timeout_ns);
                if constexpr (Q4) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t row = base + (v * 2 + s) * 256;
                        x.even = row + ((t ^ ((g & 1) << 2)) << 4);
                        x.odd = row + (((t + 4) ^ ((g & 1) << 2)) << 4);
                        float2 sx[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t sc = buf + kChunkBytes + ((nt * 8 + 2 * t) * kScales + v * 2 + s) * 4;
                            sx[nt].x = __uint_as_float(ld_shared_u1(sc));
                            sx[nt].y = __uint_as_float(ld_shared_u1(sc + kScales * 4));
                        }
                        block_q4<NT, G, Z>(acc, x, sx, ring.block() + s * 2048, ring.scales() + s * (128 / G) * 64,
                                                   ring.scales() + kScaleBytes + s * (128 / G) * 32, lane);
                    }
                } else {
                    // (a bf16 unit is half of a 128-byte row of octets)
                    x.even = base + (v >> 1) * 128 + (((t + 4 * (v & 1)) ^ ((g & 1) << 2)) << 4);
                    block_bf16<NT, LO>(acc, x, 0, ring.block(), lane);
                }
                __syncwarp();      // every lane has read the stage before it is filled again
                fetch(ring.take);
                ring.taken();
            }
        }
        n0 += warp * P::kCols;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = nt * 8 + 2 * t + j;
                if (row < rows) {
                    float* dst = part + row * ld;
                    if constexpr (Q4) {
                        const int n = n0 + 4 * column_group(g);
                        if (n < N)
                            *reinterpret_cast<float4*>(dst + n) = make_float4(acc[0][nt][j], acc[0][nt][j + 2], acc[1][nt][j], acc[1][nt][j + 2]);
                    } else {
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                const int n = n0 + mt * 16 + g + 8 * w;
                                if (n < N) dst[n] = acc[mt][nt][j + 2 * w];
                            }
                    }
                }
            }
    }

    // Goes through this CTA's items of product p; f(matrix, tile, i0, i1,
    // part number) works on a segment.
    template <class F>
    __device__ __forceinline__ void walk(int p, F f)
    {
        const Product& q = pr[p];
        for (int n = 0;; ++n) {
            const int id = item_at(q, queue[p], n, ctrl, timeout_ns);
            if (id >= q.items) return;
            int b = q.begin(id);
            const int e = q.end(id);
            while (b < e) {
                const int tile = b / q.kb, t0 = tile * q.kb, end = min(t0 + q.kb, e);
                const int matrix = tile / q.tiles;
                f(matrix, tile - matrix * q.tiles, b - t0, end - t0, id - q.item_of(t0));
                b = end;
            }
        }
    }
};

}  // namespace skinny
}  // namespace tovl
