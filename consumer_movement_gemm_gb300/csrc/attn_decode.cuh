// attn_decode.cuh -- attention of one new token per request over a paged cache.
//
//   out[b][h] = sum_t softmax_t(scale * q[b][h] . k[t]) v[t]
//
// over the last `window` (or all) of the request's tokens t, whose rows lie in
// the pages of its table.  One pass over the rows: scores, the running maximum
// m, the running sum of exp2(score - m) and the weighted rows of v, rescaled
// where m grows by more than kSlack.
//
// The rows are bytes to be streamed, each used for the group's query heads
// only, so the tensor instructions take the rows as their 16-row operand and
// the heads as the 8 columns of the other: S^T = K Q^T and O^T = V^T P^T, with
// S^T's accumulators turned into P^T's fragments by an 8 x 8 transposition in
// registers.  bf16 caches: P enters the second product as two bf16 numbers, its
// upper bits and the rest (2^-15 is left); one bf16 P would add as much error
// as the rounding of the result.  Exponentials below 2^-126 are 0.  e4m3 caches: rows become fp16 exactly, q fp16
// times a power of two per head, P times the row's scale fp16 (2^-11 of
// itself, below 2^-14 of the largest an absolute 2^-25 of that).
//
// Work: a tile is 16 to 64 rows of one key head for 8 or 16 of its query heads.
// All tiles of the call, in the order request, head, token, are shared out evenly
// to the warps of a grid that fills the GPU, whatever the lengths.  A warp streams
// its tiles through a ring of its own in shared memory, across the ends of segments
// (one request and head), without a CTA barrier; boxes of page x columns come by TMA
// (where pages are no multiples of 8 slots or short rows lie off the 32-byte
// sectors, rows by cp.async).  Segments that several warps share leave (m, sum, O)
// behind; the CTA joins its warps', and of CTAs that share a segment the last to
// finish joins theirs, in the order of the tokens, so that a call's bits depend on
// its arguments alone.
//
// What bounds it: HBM with bf16 rows (64 requests up to 16384 tokens, 8 heads of
// 128 for 32: 330 us, 6.6 TB/s; 16 of 16384, 32 heads for 32: 626 us, 6.9 TB/s),
// latency of the instructions between e4m3 row and product at three warps a
// scheduler (4 of 65536 tokens: 90 us, 6.1 TB/s; heads of 64 5.6), and for few
// tokens a chain of dependent steps: launch, lengths, shares, page, rows, products,
// parts and their joins (1 request of 64 tokens 5.1 us, of 777 8.6, of 4096 10.6).
// With eight warps instead of twelve the first takes 346 us, the third 105; with rows
// by cp.async the first took 372 us where it took 350 with boxes.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "common.cuh"
#include "paged.cuh"
#include "sync.cuh"

namespace tovl {
namespace attn {

// PAIR: two warps take two blocks of the same key head's query heads from one ring.
template <int DP_, bool F8_, int NT_, bool PAIR_ = false>
struct Shape {
    static constexpr int DP = DP_;                 // head dimension, filled up
    static constexpr bool F8 = F8_;
    static constexpr int NT = NT_;                 // blocks of 8 query heads
    static constexpr int kRingLog = PAIR_ ? 1 : 0;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kBlockRow = DP * (F8 ? 1 : 2) > 64 ? 128 : 64;            // bytes of a row in a column block
    static constexpr int CB = (DP * (F8 ? 1 : 2) + kBlockRow - 1) / kBlockRow;
    static constexpr int kRow = CB * kBlockRow;
    static constexpr int kTile = kRow <= 64 ? 64 : kRow <= 128 ? 32 : 16;
    static constexpr int kBlock = kTile * kBlockRow;
    static constexpr int kRows = CB * kBlock;      // all of k or of v
    static constexpr int MT = kTile / 16;
    static constexpr int JT = DP / 16;             // blocks of 16 columns
    static constexpr int kStage = 2 * kRows;
    static constexpr int kScaleStage = F8 ? 2 * kTile * 4 : 0;
    // e4m3 with two blocks of heads: twelve warps of 168 registers (64 and 128 columns
    // spill 16 and 104 bytes a thread), eight of 255 (256 columns: 8 bytes).
    static constexpr int kWarps = kRow > 384 && !PAIR_ ? 6 : kRow > 256 && !PAIR_ ? 8 : NT == 1 || (F8 && DP <= 128) ? 12 : 8;
    static constexpr int kFit = (214 * 1024) / (kWarps * (kStage + kScaleStage));
    static constexpr int kStages = kFit > 4 ? 4 : kFit;                 // a warp's share of its ring's
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kScales = kStages * kScaleStage;               // of a warp, behind all rings
    static constexpr int kSmem = kWarps * (kRing + kScales) + 1024;
    static constexpr int kFrag = NT * JT * 32;     // float4 of one O
    static constexpr int kPart = kFrag * 4 + 2 * kHeads;               // floats of a part: O, m, sum
    // the 16-byte pieces of row r of a block are exchanged by XOR with this
    // (so that 8 rows' pieces lie in different banks; the copies' swizzle)
    static __host__ __device__ constexpr int phase(int r) { return kBlockRow == 128 ? r & 7 : (r >> 1) & 3; }
    static_assert(kSmem + 12 * 1024 <= 227 * 1024, "shared memory, with what is static");
    static_assert(kStages << kRingLog >= 2 && kBlock % 1024 == 0 && kPart * 4 <= kRing, "ring");
};

// What is left behind of a segment that does not lie within one warp's share.
struct Open {
    const float* part;
    int first, end;            // its tiles in the order of the call; end == 0: none
    int b, head0, n_heads;     // its request and query heads
    int beside;                // which of the heads that go together
};

// A segment whose parts are joined.
struct Joined {
    float* to;                 // where the joined part goes; null: it is the result
    int entry, n;              // its parts in the CTA's list
    int b, head0, n_heads;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Parts lie in shared memory or in the workspace, where another SM may have written them.
__device__ __forceinline__ float2 ld_part(const float2* p)
{
    float2 v;
    asm volatile("ld.relaxed.gpu.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_part(const float4* p)
{
    float4 v;
    asm volatile("ld.relaxed.gpu.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
    return v;
}
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One box of a cache: `cols` columns of one head, `rows` slots of one page.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void load_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Bounded wait for a stage's copies (a bound against logic errors).
__device__ __forceinline__ bool wait_full(uint64_t* bar, uint32_t parity, const AttnParams& p)
{
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t start = ptx::globaltimer();
    for (uint32_t i = 1; !ptx::mbar_try_wait(bar, parity); ++i) {
        if ((i & 255) == 0 && ptx::globaltimer() - start > static_cast<uint64_t>(p.timeout_ns)) {
            record_error(p.ctrl, kErrTimeout);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <bool HALF>
__device__ __forceinline__ void mma(float4& d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (HALF) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d.x), "+f"(d.y), "+f"(d.z), "+f"(d.w)
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d.x), "+f"(d.y), "+f"(d.z), "+f"(d.w)
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// four e4m3 numbers, the lower two and the upper two (exactly)
__device__ __forceinline__ void e4m3_to_h2(uint32_t four, uint32_t& lower, uint32_t& upper)
{
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }" : "=r"(lower), "=r"(upper) : "r"(four));
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// What the upper half of a weight's bits leaves.  It has the weight's sign even
// where nothing is left, so that both products with an infinite value have too.
__device__ __forceinline__ float rest(float w) { return fmaxf(w - bf_hi(__float_as_uint(w)), w * 0x1p-30f); }

// The weight of e4m3 rows is exp2(score - m) times the row's scale, m the
// largest score + log2(scale), so that the product's operand is 2^kSlack at most.  The
// sum takes the same exponential without the scale, 2^(kShift + kSlack) / scale at most.
// Smaller scales than 2^kLeastScale count as that in m, so a term is below 2^97 and the
// sum of 2^31 inside fp32; 1e-12 / 448, the least that rope_append writes, is above it.
// The shift keeps the terms of large scales: of 2^127 down to 2^-39 of the largest.
constexpr float kShift = 40.f;
constexpr float kLeastScale = -48.75f;

// A score may be over the maximum that weights are taken relative to by this much
// (weights up to 256) before it becomes the maximum: a tile then costs one vote,
// not a reduction over the rows for each head.
constexpr float kSlack = 8.f;

// First tile and number of tiles of a request.
template <int TILE>
__device__ __forceinline__ int tiles_of(const AttnParams& p, int len, int& first)
{
    const int lo = p.window && len > p.window ? len - p.window : 0;
    first = lo / TILE;
    return len > 0 ? (len - 1) / TILE + 1 - first : 0;
}

// (p.most_tokens: what a table's row holds, and tiles of whole int positions)
__device__ __forceinline__ int length_of(const AttnParams& p, int b)
{
    return min(max(__ldg(p.length + b), 0), p.most_tokens);
}

// a / b.  Below 2^20 (a + 1/2) / b is at least 1 / (2 b) from a whole number, and the
// quotient of floats off by 1 / (4 b) at most.
__device__ __forceinline__ int quotient(int a, int b)
{
    return a < 1 << 20 ? static_cast<int>(__fdividef(a + 0.5f, static_cast<float>(b))) : a / b;
}

// A place in the order of the call: request, key head, block of its query
// heads, tile.
template <class S>
struct Cursor {
    int left;                  // tiles of the share from here on
    int b, vh, head, block, tile;
    int len, first, count;     // of the request

    __device__ __forceinline__ void enter(const AttnParams& p)
    {
        len = length_of(p, b);
        count = tiles_of<S::kTile>(p, len, first);
    }
    __device__ __forceinline__ void at_head(int v, int per_head)
    {
        vh = v;
        head = per_head == 1 ? v : quotient(v, per_head);
        block = v - head * per_head;
    }
    // together: blocks of heads that neighbouring warps take side by side
    __device__ __forceinline__ void next(const AttnParams& p, int per_head, int together)
    {
        --left;
        if (++tile < first + count || left == 0) return;
        const int heads = p.cache.heads * per_head, v = vh + together;
        if (v >= heads) {
            at_head(v - heads, per_head);
            do {
                ++b;
                enter(p);
            } while (count == 0);       // (a share ends at the last request with tiles)
        } else {
            at_head(v, per_head);
        }
        tile = first;
    }
};

// What a sum of weights divides: 1 / l, without the shift.  (__fdividef is 0 from 2^126 on.)
template <class S>
__device__ __forceinline__ float over(float l)
{
    if (l == 0.f) return 0.f;
    return S::F8 ? __fdividef(0x1p8f, l * 0x1p-32f) : __fdividef(1.f, l);
}

// Stores float4 j of a lane's O^T, times i0 and i1 (its two heads'): rows of out
// from `out` on.  x and z are of head 2 (lane % 4), y and w of the next; x and y of
// one column, z and w of the next (e4m3) or the eighth after it, whose lanes
// exchange numbers for pairs of columns.  All lanes of a warp.
template <class S>
__device__ __forceinline__ void store_pair(__nv_bfloat16* out, int dim, int heads, int j, int lane, float4 o, float i0, float i1)
{
    const int g = lane >> 2, h = 2 * (lane & 3);
    if constexpr (S::F8) {
        const int d = 16 * j + 2 * g;
        if (d >= dim) return;
        if (h < heads) *reinterpret_cast<uint32_t*>(out + h * dim + d) = ptx::pack_bf16x2(o.x * i0, o.z * i0);
        if (h + 1 < heads) *reinterpret_cast<uint32_t*>(out + (h + 1) * dim + d) = ptx::pack_bf16x2(o.y * i1, o.w * i1);
    } else {
        const bool odd = g & 1;
        const uint32_t a = ptx::pack_bf16x2(o.x * i0, o.z * i0), b = ptx::pack_bf16x2(o.y * i1, o.w * i1);
        const uint32_t mine = odd ? b : a, other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 4);
        const int d = 16 * j + (g & ~1), row = h + (odd ? 1 : 0);
        if (row >= heads) return;
        out += row * dim + d;
        if (d < dim) *reinterpret_cast<uint32_t*>(out) = odd ? __byte_perm(other, mine, 0x5410) : __byte_perm(mine, other, 0x5410);
        if (d + 8 < dim) *reinterpret_cast<uint32_t*>(out + 8) = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x7632);
    }
}

template <class S>
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.f ? -INFINITY : (m + lg2(l) - (S::F8 ? kShift : 0.f)) * 0.693147180559945309f;
}

// Sums of tiles stop there.
constexpr unsigned kMostTiles = 0x7fffffffu;

// CTAs that share a segment join in groups of kGroup where there are more than kFlat.
constexpr int kFlat = 24;
constexpr int kGroup = 12;
constexpr int kAtOnce = 4;     // segments of other CTAs that are joined at a time

// What each CTA gets of the call's tiles: `each`, the first `rest` one more; or,
// where all segments have as many tiles, one of `parts` parts of one of them,
// shared out alike.
struct Shares {
    int ctas, each, rest;
    int parts;                 // 0: the former
    __device__ __forceinline__ int start(int c) const { return c * each + min(c, rest); }
    // the CTA that a tile belongs to
    __device__ __forceinline__ int owner(int tile) const
    {
        const int longer = rest * (each + 1);
        return tile < longer ? quotient(tile, each + 1) : rest + quotient(tile - longer, each);
    }
};

// U float4 of O^T of a segment's parts, 32 apart, joined in their order, six at a time:
// the sums relative to the largest m of their two heads (x and z are of one, y and w of
// the other).  The sums do not depend on U.
template <int U>
__device__ __forceinline__ void join(const float* const* part, int n, int stats, int sums, int e, float4 (&o)[U], float2& m, float2& l)
{
    constexpr int kAhead = 6;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < U; ++u) o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    m = make_float2(-INFINITY, -INFINITY), l = make_float2(0.f, 0.f);
    for (int i = 0; i < n; i += kAhead) {
        // m and l of each part, then the weights; U > 1: a lane's each, of part lane / 4
        // and heads 2 (lane % 4)
        constexpr int kOwn = U == 1 ? kAhead : 1;
        float2 w[kOwn], s[kOwn];
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int which = U == 1 ? k : lane / 4;
            w[k] = make_float2(-INFINITY, -INFINITY), s[k] = make_float2(0.f, 0.f);
            if (which >= kAhead || i + which >= n) continue;
            const float* const q = part[i + which] + stats;
            w[k] = ld_part(reinterpret_cast<const float2*>(q)), s[k] = ld_part(reinterpret_cast<const float2*>(q + sums));
        }
        float4 v[kAhead][U];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v[k][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i + k < n) v[k][u] = ld_part(reinterpret_cast<const float4*>(part[i + k]) + e + u * 32);
            }
        const float2 was = m;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) m.x = fmaxf(m.x, w[k].x), m.y = fmaxf(m.y, w[k].y);
        if (U > 1)
#pragma unroll
            for (int d = 4; d < 32; d *= 2) m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, d)), m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, d));
        const float u0 = m.x == -INFINITY ? 0.f : m.x, u1 = m.y == -INFINITY ? 0.f : m.y;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) w[k].x = ex2(w[k].x - u0), w[k].y = ex2(w[k].y - u1);
        if (i) {
            const float c0 = ex2(was.x - u0), c1 = ex2(was.y - u1);
            l.x *= c0, l.y *= c1;
#pragma unroll
            for (int u = 0; u < U; ++u) o[u].x *= c0, o[u].y *= c1, o[u].z *= c0, o[u].w *= c1;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            float2 wk = w[k % kOwn], sk = s[k % kOwn];
            if (U > 1) {
                const int from = k * 4 + (lane & 3);
                wk.x = __shfl_sync(0xffffffffu, wk.x, from), wk.y = __shfl_sync(0xffffffffu, wk.y, from);
                sk.x = __shfl_sync(0xffffffffu, sk.x, from), sk.y = __shfl_sync(0xffffffffu, sk.y, from);
            }
            l.x = fmaf(sk.x, wk.x, l.x), l.y = fmaf(sk.y, wk.y, l.y);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                o[u].x = fmaf(v[k][u].x, wk.x, o[u].x), o[u].y = fmaf(v[k][u].y, wk.y, o[u].y);
                o[u].z = fmaf(v[k][u].z, wk.x, o[u].z), o[u].w = fmaf(v[k][u].w, wk.y, o[u].w);
            }
        }
    }
}

// The segments of a list, U column blocks of 16 of 8 heads a warp.
template <class S, int U>
__device__ __forceinline__ void join_all(const AttnParams& p, const Joined* joined, const float* const* parts, int count, int warp, int lane)
{
    static_assert(S::JT % U == 0, "every column block of a segment is one warp's");
    constexpr int kOfHeads = S::JT / U, kUnits = S::NT * kOfHeads;
    for (int at = warp; at < count * kUnits; at += S::kWarps) {
        const Joined seg = joined[at / kUnits];
        const int nt = at % kUnits / kOfHeads, j0 = at % kOfHeads * U, e = (nt * S::JT + j0) * 32 + lane, h = nt * 8 + 2 * (lane & 3);
        float2 m, l;
        float4 sum[U];
        join<U>(parts + seg.entry, seg.n, S::kFrag * 4 + h, S::kHeads, e, sum, m, l);
        const bool stats = j0 == 0 && lane < 4;
        if (seg.to) {
#pragma unroll
            for (int u = 0; u < U; ++u) reinterpret_cast<float4*>(seg.to)[e + u * 32] = sum[u];
            if (stats) {
                *reinterpret_cast<float2*>(seg.to + S::kFrag * 4 + h) = m;
                *reinterpret_cast<float2*>(seg.to + S::kFrag * 4 + S::kHeads + h) = l;
            }
        } else {
            __nv_bfloat16* const row = static_cast<__nv_bfloat16*>(p.out) + seg.b * p.ldo + static_cast<long long>(seg.head0 + nt * 8) * p.cache.dim;
            const float i0 = over<S>(l.x), i1 = over<S>(l.y);
#pragma unroll
            for (int u = 0; u < U; ++u) store_pair<S>(row, p.cache.dim, seg.n_heads - nt * 8, j0 + u, lane, sum[u], i0, i1);
            if (stats && p.lse) {
                float* const lse = p.lse + static_cast<long long>(seg.b) * p.Hq + seg.head0;
                if (h < seg.n_heads) lse[h] = lse_of<S>(m.x, l.x);
                if (h + 1 < seg.n_heads) lse[h + 1] = lse_of<S>(m.y, l.y);
            }
        }
    }
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1) attn_decode_kernel(const __grid_constant__ AttnParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_full[S::kWarps * S::kStages], s_empty[S::kWarps * S::kStages];
    __shared__ int4 s_meta[S::kWarps * S::kStages];
    constexpr int kEntries = kAtOnce * kFlat > 2 * S::kWarps ? kAtOnce * kFlat : 2 * S::kWarps;
    __shared__ unsigned s_sum[S::kWarps], s_upto[S::kThreads];
    __shared__ int s_flags[S::kWarps];
    __shared__ Open s_open[S::kWarps * 2];
    __shared__ const float* s_part[kEntries];
    __shared__ Joined s_joined[S::kWarps * 2];
    __shared__ uint32_t s_won;
    constexpr int kTile = S::kTile, NT = S::NT, JT = S::JT, MT = S::MT, kStages = S::kStages, CB = S::CB;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0 && p.boxed) {
        ptx::prefetch_tmap(&p.k_map);
        ptx::prefetch_tmap(&p.v_map);
    }
    constexpr int kRingLog = S::kRingLog, kRingStages = kStages << kRingLog;
    if (lane < kStages) ptx::mbar_init(&s_full[warp * kStages + lane], 1), ptx::mbar_init(&s_empty[warp * kStages + lane], 1 << kRingLog);
    if (lane < 2) s_open[warp * 2 + lane].end = 0;
    ptx::fence_mbar_init();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    // ---------------------------------------------------------------- shares
    const int per_head = (p.group + S::kHeads - 1) / S::kHeads, together = 1 << p.together_log;
    const int groups = p.cache.heads * per_head >> p.together_log;
    const int beside = warp & (together - 1), turn = warp >> p.together_log, turns = S::kWarps >> p.together_log;
    const int chunk = (p.B + S::kThreads - 1) / S::kThreads, b0 = tid * chunk;
    int unused;
    const int first_count = tiles_of<kTile>(p, length_of(p, 0), unused);
    unsigned upto = 0;                       // tiles of a head, of requests up to this thread's; the sums stop at the most
    bool none = false, equal = true;
    for (int b = b0; b < min(p.B, b0 + chunk); ++b) {
        const int len = __ldg(p.length + b);
        if (len < 0 || len > p.most_tokens) record_error(p.ctrl, kErrInvalid);
        const int count = tiles_of<kTile>(p, length_of(p, b), unused);
        upto = min(upto + count, kMostTiles);
        none |= len <= 0;
        equal &= count == first_count;
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const unsigned o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto = min(upto + o, kMostTiles);
    }
    s_upto[tid] = upto;
    none = __any_sync(0xffffffffu, none), equal = __all_sync(0xffffffffu, equal);
    if (lane == 31) s_sum[warp] = upto, s_flags[warp] = (none ? 1 : 0) | (equal ? 0 : 2);
    __syncthreads();
    unsigned sums = lane < S::kWarps ? s_sum[lane] : 0;       // of the warps up to `lane`
    const int flag = lane < S::kWarps ? s_flags[lane] : 0;
#pragma unroll
    for (int d = 1; d < S::kWarps; d *= 2) {
        const unsigned o = __shfl_up_sync(0xffffffffu, sums, d);
        if (lane >= d) sums = min(sums + o, kMostTiles);
    }
    none = __any_sync(0xffffffffu, flag & 1), equal = !__any_sync(0xffffffffu, flag & 2);
    const unsigned all = __shfl_sync(0xffffffffu, sums, S::kWarps - 1);
    if (all > p.most_tiles) {
        if (tid == 0) record_error(p.ctrl, kErrUnsupported);
        return;
    }
    const int total = all * groups, cta = blockIdx.x;
    // CTAs that get work: all, but with few tiles, in segments of one length, a multiple
    // of the segments, so that none of them reaches into two.  A segment of up to three
    // tiles a warp is one CTA's, because the join of CTAs costs more than two tiles; a
    // longer one is split to a tile a warp, and from the twelfth CTA on to two, where more
    // parts to join cost as much as they save.  One request, 8 heads: 300 tokens in one
    // CTA a head 7.0 us, in equal parts over all CTAs 9.4; 777 in five 8.6, over all 10.7;
    // 4096 in 12 10.6, over all 12.1.
    Shares shares = {static_cast<int>(gridDim.x), 0, 0, 0};
    const int grid = gridDim.x, segments = p.B * groups;
    if (equal && segments <= grid && total < 4 * grid * turns) {
        const int most = p.by_turns.div(first_count + turns - 1);
        const int want = most <= 3 ? 1 : max(min(most, 12), (most + 1) / 2);
        const int parts = min(want, quotient(grid, segments));
        if (parts == want || segments * parts * 5 >= grid * 4) shares.parts = parts, shares.ctas = segments * parts;
    }
    // requests without tokens: nothing of theirs is in the order
    for (int b = blockIdx.x; none && b < p.B; b += gridDim.x) {
        if (__ldg(p.length + b) > 0) continue;
        uint4* const out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + b * p.ldo);
        for (int i = tid; i < p.Hq * p.cache.dim / 8; i += S::kThreads) out[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = tid; i < p.Hq; i += S::kThreads) p.lse[static_cast<long long>(b) * p.Hq + i] = -INFINITY;
    }
    if (total == 0 || cta >= shares.ctas) return;
    int whole = total, among = shares.ctas, place = cta, offset = 0;
    if (shares.parts) {
        const int segment = quotient(cta, shares.parts);
        whole = first_count, among = shares.parts, place = cta - segment * shares.parts, offset = segment * first_count;
    }
    shares.each = quotient(whole, among), shares.rest = whole - shares.each * among;
    const int cta_from = offset + shares.start(place), cta_to = offset + shares.start(place + 1);

    // this warp's share, and the request that its first tile lies in
    Cursor<S> put;
    int warp_from;
    {
        const int n = cta_to - cta_from, each = p.by_turns.div(n), rest = n - each * turns;
        put.left = each + (turn < rest ? 1 : 0);
        warp_from = cta_from + turn * each + min(turn, rest);
    }
    if (put.left > 0) {
        const unsigned tile = p.by_groups.div(warp_from);
        const int w = __popc(__ballot_sync(0xffffffffu, lane < S::kWarps && sums <= tile));
        const unsigned base = w ? __shfl_sync(0xffffffffu, sums, w - 1) : 0, reach = base + s_upto[min(w, S::kWarps - 1) * 32 + lane];
        const int i = __popc(__ballot_sync(0xffffffffu, reach <= tile));
        const unsigned start = __shfl_sync(0xffffffffu, reach, max(i - 1, 0));
        int r = warp_from - (i ? start : base) * groups;
        for (put.b = (w * 32 + i) * chunk;; ++put.b) {
            put.enter(p);
            if (r < put.count * groups) break;
            r -= put.count * groups;
        }
        const int group = quotient(r, put.count);
        put.at_head(group * together + beside, per_head);
        put.tile = put.first + r - group * put.count;
    }

    // ---------------------------------------------------------------- a warp's stream
    const int owner = warp >> kRingLog << kRingLog;      // the ring's first warp, which fetches
    uint8_t* const rings = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* const ring = rings + owner * S::kRing;
    uint8_t* const ring_scales = rings + S::kWarps * S::kRing + owner * S::kScales;
    uint64_t *const full = s_full + owner * kStages, *const empty = s_empty + owner * kStages;
    int4* const metas = s_meta + owner * kStages;
    const uint32_t ring_u = ptx::smem_u32(ring), scales_u = ptx::smem_u32(ring_scales);
    const int tiles = put.left;
    // boxes: lane (k or v, column block, piece of the tile's rows)
    const int pieces_log = p.pieces_log, box_rows = kTile >> pieces_log;
    const int piece = lane & ((1 << pieces_log) - 1), box_col = (lane >> pieces_log) % CB, box_kv = (lane >> pieces_log) / CB;
    const uint32_t box_at = box_kv * S::kRows + box_col * S::kBlock + piece * box_rows * S::kBlockRow;
    // what the next tile needs from this lane: a box's page and first slot, or (rows
    // one by one) those of the rows lane and lane + 32
    constexpr int kOwn = kTile > 32 ? 2 : 1;
    int page_id[kOwn], page_in[kOwn];
    const auto find_pages = [&]() {
        const int lo = p.window && put.len > p.window ? put.len - p.window : 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int row = p.boxed ? piece * box_rows : i * 32 + lane, t = put.tile * kTile + row, rows = p.boxed ? box_rows : 1;
            page_id[i] = -1;
            if (put.left > 0 && row < kTile && t < put.len && t + rows > lo) {
                const int n = p.by_page.div(t);
                page_in[i] = t - n * p.cache.page;
                page_id[i] = __ldg(p.table + put.b * p.ldt + n);
                if (static_cast<unsigned>(page_id[i]) >= static_cast<unsigned>(p.cache.pages)) page_id[i] = -2;
            }
        }
    };
    // starts the copies of the tile at `put` and moves on
    const auto fetch = [&](int stage) {
        if (put.left > 0) {
            const uint32_t dst = ring_u + stage * S::kStage;
            const int head = put.head;
            if (lane == 0) {
                const int last = put.first + put.count - 1;
                metas[stage] = make_int4(put.b, put.head | put.block << 16, put.tile | (put.tile == put.first ? 1 << 30 : 0) | (put.tile == last ? 1 << 31 : 0), put.len);
            }
            if (page_id[0] == -2 || page_id[kOwn - 1] == -2) record_error(p.ctrl, kErrInvalid);
            if (p.boxed) {
                // what holds no token of this tile is outside the tensor: zeros, and nothing read
                const uint32_t bar = ptx::smem_u32(full + stage);
                const bool in = page_id[0] >= 0;
                uint32_t bytes = 2 * S::kRows;
                if (S::F8) bytes += 8 * box_rows * __popc(__ballot_sync(0xffffffffu, in && lane < 1 << pieces_log));
                if (lane == 0) ptx::mbar_arrive_expect_tx(full + stage, bytes);
                if (lane < 2 * CB << pieces_log) {
                    const int x = box_col * (S::kBlockRow / (S::F8 ? 1 : 2)), page = in ? page_id[0] : p.cache.pages, slot = in ? page_in[0] : 0;
                    load_box(dst + box_at, box_kv ? &p.v_map : &p.k_map, bar, x, p.slots_first ? slot : head, p.slots_first ? head : slot, page);
                    if (S::F8 && in && box_col == 0) {
                        const long long at = (static_cast<long long>(page) * p.cache.heads + head) * p.cache.page + slot;
                        load_bulk(scales_u + stage * S::kScaleStage + (box_kv * kTile + piece * box_rows) * 4, (box_kv ? p.cache.v_scale : p.cache.k_scale) + at,
                                  box_rows * 4, bar);
                    }
                }
            } else {
                long long off[kOwn];
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    off[i] = -1;
                    if (page_id[i] >= 0) {
                        off[i] = page_id[i] * p.cache.page_stride + page_in[i] * p.cache.slot_stride + head * p.cache.head_stride;
                        if (S::F8) {
                            const long long at = (static_cast<long long>(page_id[i]) * p.cache.heads + head) * p.cache.page + page_in[i];
                            cp_async4(scales_u + stage * S::kScaleStage + (i * 32 + lane) * 4, p.cache.k_scale + at, 4);
                            cp_async4(scales_u + stage * S::kScaleStage + (kTile + i * 32 + lane) * 4, p.cache.v_scale + at, 4);
                        }
                    }
                }
                constexpr int kPerRow = S::kRow / 16, kPerBlock = S::kBlockRow / 16;
                const int bytes = p.cache.dim * (S::F8 ? 1 : 2);
#pragma unroll
                for (int i = 0; i < kTile * kPerRow / 32; ++i) {
                    static_assert(kOwn == 1 || 32 % kPerRow == 0, "rows of one instruction lie in one lane's part");
                    const int row = (i * 32 + lane) / kPerRow, c = (i * 32 + lane) % kPerRow;
                    const long long o = __shfl_sync(0xffffffffu, off[kOwn == 1 ? 0 : i * 32 / kPerRow / 32], row & 31);
                    const bool in = o >= 0 && c * 16 < bytes;
                    const long long src = in ? o + c * 16 : 0;
                    const uint32_t at = dst + c / kPerBlock * S::kBlock + row * S::kBlockRow + ((c % kPerBlock ^ S::phase(row)) << 4);
                    cp_async16(at, p.cache.k + src, in ? 16 : 0);
                    cp_async16(at + S::kRows, p.cache.v + src, in ? 16 : 0);
                }
            }
            put.next(p, per_head, together);
            find_pages();
        }
        cp_commit();
    };
    if (tiles > 0) {
        if (warp == owner) {
            find_pages();
#pragma unroll
            for (int s = 0; s < kRingStages; ++s) fetch(s);
        }
        // fragments of k: row lane % 16, 16 bytes lane / 16; of v: the same (e4m3),
        // or row lane % 8 + 8 (lane / 16), 16 bytes lane / 8 % 2
        const int k_row = lane & 15, v_row = S::F8 ? k_row : (lane & 7) + (lane >> 4) * 8;
        const uint32_t k_base = k_row * S::kBlockRow, v_base = v_row * S::kBlockRow;
        const uint32_t k_turn = ((lane >> 4) ^ S::phase(k_row)) << 4, v_turn = ((S::F8 ? lane >> 4 : (lane >> 3) & 1) ^ S::phase(v_row)) << 4;
        // 16-byte piece c (even; the lanes add the last bit) of 16 rows from row `row` on
        const auto piece_at = [](uint32_t base, uint32_t turn, int row, int c) {
            return base + c / (S::kBlockRow / 16) * S::kBlock + row * S::kBlockRow + (turn ^ (c % (S::kBlockRow / 16) << 4));
        };

        float4 o[NT][JT];
        uint32_t q[NT][JT][2];
        float m[NT][2], l[NT][2], q_unit[NT][2];
        int seg_first = 0;
        bool began = false, fresh = true;
        int stage = 0;
        uint32_t parity = 0;
        for (int it = 0; it < tiles; ++it) {
            const auto wait = [&]() {
                if (!p.boxed) {
                    if (it) cp_wait<kRingStages - 2>();
                    else cp_wait<kRingStages - 1>();
                    return true;
                }
                if (wait_full(full + stage, parity, p)) return true;
                // the other copies in flight, then out
                for (int s = 1; s < kRingStages - (it ? 1 : 0) && it + s < tiles; ++s) {
                    if (++stage == kRingStages) stage = 0, parity ^= 1;
                    wait_full(full + stage, parity, p);
                }
                return false;
            };
            __syncwarp();
            // (a shared ring's other warps learn of a tile by its arrival)
            if (kRingLog && !wait()) break;
            const int4 meta = metas[stage];
            const int b = meta.x, tile = meta.z & 0x3fffffff, len = meta.w;
            const int block = (meta.y >> 16) + (kRingLog ? beside & 1 : 0), head0 = (meta.y & 0xffff) * p.group + block * S::kHeads, n_heads = min(S::kHeads, p.group - block * S::kHeads);
            if (fresh) {
                // the segment's queries
                fresh = false;
                began = meta.z & (1 << 30);
                int f;
                tiles_of<kTile>(p, len, f);
                seg_first = warp_from + it - (tile - f);
                const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q) + b * p.ldq;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    // (columns behind the last head repeat it, and their results are dropped)
                    const int h = min(nt * 8 + (lane >> 2), n_heads - 1);
                    const __nv_bfloat16* row = qp + static_cast<long long>(head0 + h) * p.cache.dim + (S::F8 ? 4 : 2) * (lane & 3);
                    float top = 0.f;
#pragma unroll
                    for (int j = 0; j < JT; ++j) {
                        if constexpr (S::F8) {
                            const uint2 u = 16 * j < p.cache.dim ? __ldg(reinterpret_cast<const uint2*>(row + 16 * j)) : make_uint2(0, 0);
                            q[nt][j][0] = u.x, q[nt][j][1] = u.y;
                            top = fmaxf(top, fmaxf(fmaxf(fabsf(bf_lo(u.x)), fabsf(bf_hi(u.x))), fmaxf(fabsf(bf_lo(u.y)), fabsf(bf_hi(u.y)))));
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int d = 16 * j + 8 * i;
                                q[nt][j][i] = d < p.cache.dim ? __ldg(reinterpret_cast<const uint32_t*>(row + d)) : 0u;
                            }
                        }
                    }
                    if constexpr (S::F8) {
                        // fp16 times the power of two that brings the row's largest to [2^14, 2^15)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112), 127);
                        const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
#pragma unroll
                        for (int j = 0; j < JT; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) q[nt][j][i] = pack_h2(bf_lo(q[nt][j][i]) * up, bf_hi(q[nt][j][i]) * up);
                        const float down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * p.scale_log2;
                        q_unit[nt][0] = __shfl_sync(0xffffffffu, down, 8 * (lane & 3));
                        q_unit[nt][1] = __shfl_sync(0xffffffffu, down, 8 * (lane & 3) + 4);
                    } else {
                        q_unit[nt][0] = q_unit[nt][1] = p.scale_log2;
                    }
                    m[nt][0] = m[nt][1] = -INFINITY;
                    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                    for (int j = 0; j < JT; ++j) o[nt][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            if (!kRingLog && !wait()) break;
            __syncwarp();
            if (it && warp == owner) {
                // into the stage of the tile before, when the ring's warps are through with it.
                // (Right behind that tile more copies are in flight, and memory is slower:
                // 64 requests up to 16384 tokens 343 us for 330.)
                const int to = stage == 0 ? kRingStages - 1 : stage - 1;
                if (kRingLog && put.left > 0 && !wait_full(empty + to, stage == 0 ? parity ^ 1 : parity, p)) put.left = 0;
                fetch(to);
            }
            uint8_t* const st = ring + stage * S::kStage;
            const uint32_t st_u = ring_u + stage * S::kStage;

            // scores: rows lane / 4 and + 8 of each 16, heads 2 (lane % 4) and + 1
            float4 s[NT][MT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) s[nt][mt] = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t k_at = st_u + k_base;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (S::F8) {
#pragma unroll
                    for (int j = 0; j < JT; j += 2) {
                        uint32_t a[4];
                        ldsm(a, piece_at(k_at, k_turn, mt * 16, j));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t a0, a1, a2, a3;
                            e4m3_to_h2(a[2 * i], a0, a2);
                            e4m3_to_h2(a[2 * i + 1], a1, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma<true>(s[nt][mt], a0, a1, a2, a3, q[nt][j + i][0], q[nt][j + i][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < JT; ++j) {
                        uint32_t a[4];
                        ldsm(a, piece_at(k_at, k_turn, mt * 16, 2 * j));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma<false>(s[nt][mt], a[0], a[1], a[2], a[3], q[nt][j][0], q[nt][j][1]);
                    }
                }
            }
            // rows of this tile that count
            const int lo = (p.window && len > p.window ? len - p.window : 0) - tile * kTile, hi = len - tile * kTile;
            const bool partial = lo > 0 || hi < kTile;
            const float* scales = reinterpret_cast<const float*>(ring_scales + stage * S::kScaleStage);
            float vs[MT][2], vl[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = mt * 16 + i * 8 + (lane >> 2);
                    float ks = 1.f;
                    vs[mt][i] = 1.f, vl[mt][i] = 0.f;
                    if (S::F8) {
                        ks = scales[r];
                        vs[mt][i] = scales[kTile + r] * 0x1p-40f;
                        vl[mt][i] = fmaxf(lg2(scales[kTile + r]), kLeastScale);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float& x = i ? s[nt][mt].z : s[nt][mt].x;
                        float& y = i ? s[nt][mt].w : s[nt][mt].y;
                        x *= q_unit[nt][0] * ks;
                        y *= q_unit[nt][1] * ks;
                    }
                }
            if (partial) {
                // other rows (of this page, or zeros) have no weight, and no value that a weight of 0 could not stand
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = mt * 16 + i * 8 + (lane >> 2);
                        if (r >= lo && r < hi) continue;
                        vs[mt][i] = vl[mt][i] = 0.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (i) s[nt][mt].z = s[nt][mt].w = -INFINITY;
                            else s[nt][mt].x = s[nt][mt].y = -INFINITY;
                        }
                    }
                for (int i = lane; i < S::kRows / 16; i += 32) {
                    const int r = i * 16 % S::kBlock / S::kBlockRow;
                    if (r < lo || r >= hi) *reinterpret_cast<uint4*>(st + S::kRows + i * 16) = make_uint4(0, 0, 0, 0);
                }
                // (before the copies that come to this stage next)
                ptx::fence_proxy_async_smem();
                __syncwarp();
            }
            // the maximum so far stays where no score is over it by more than kSlack
            float top[NT][2];
            bool over_it = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    top[nt][0] = fmaxf(top[nt][0], fmaxf(s[nt][mt].x + vl[mt][0], s[nt][mt].z + vl[mt][1]));
                    top[nt][1] = fmaxf(top[nt][1], fmaxf(s[nt][mt].y + vl[mt][0], s[nt][mt].w + vl[mt][1]));
                }
                over_it |= top[nt][0] > m[nt][0] + kSlack || top[nt][1] > m[nt][1] + kSlack;
            }
            if (__any_sync(0xffffffffu, over_it)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v = top[nt][i];
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                        v = fmaxf(v, m[nt][i]);
                        const float c = m[nt][i] == -INFINITY ? 0.f : ex2(m[nt][i] - v);
                        m[nt][i] = v;
                        l[nt][i] *= c;
#pragma unroll
                        for (int j = 0; j < JT; ++j) {
                            if (i) o[nt][j].y *= c, o[nt][j].w *= c;
                            else o[nt][j].x *= c, o[nt][j].z *= c;
                        }
                    }
            }
            uint32_t ph[NT][MT][2], pl[NT][MT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // (all scores -inf so far: weights of 0)
                const float u0 = (m[nt][0] == -INFINITY ? 0.f : m[nt][0]) - (S::F8 ? kShift : 0.f), u1 = (m[nt][1] == -INFINITY ? 0.f : m[nt][1]) - (S::F8 ? kShift : 0.f);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float4& v = s[nt][mt];
                    v.x = ex2(v.x - u0), v.y = ex2(v.y - u1), v.z = ex2(v.z - u0), v.w = ex2(v.w - u1);
                    l[nt][0] += v.x + v.z, l[nt][1] += v.y + v.w;
                    if constexpr (S::F8) {
                        ph[nt][mt][0] = transpose8(pack_h2(v.x * vs[mt][0], v.y * vs[mt][0]));
                        ph[nt][mt][1] = transpose8(pack_h2(v.z * vs[mt][1], v.w * vs[mt][1]));
                    } else {
                        ph[nt][mt][0] = transpose8(__byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632));
                        ph[nt][mt][1] = transpose8(__byte_perm(__float_as_uint(v.z), __float_as_uint(v.w), 0x7632));
                        pl[nt][mt][0] = transpose8(ptx::pack_bf16x2(rest(v.x), rest(v.y)));
                        pl[nt][mt][1] = transpose8(ptx::pack_bf16x2(rest(v.z), rest(v.w)));
                    }
                }
            }
            // O^T += V^T P^T
            const uint32_t v_at = st_u + S::kRows + v_base;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (S::F8) {
#pragma unroll
                    for (int j = 0; j < JT; j += 2) {
                        uint32_t a[4];
                        ldsm_t(a, piece_at(v_at, v_turn, mt * 16, j));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // bytes: row 0's columns 0, 1, row 1's -> column 0 of both rows, column 1 of both
                            uint32_t a0, a1, a2, a3;
                            e4m3_to_h2(__byte_perm(a[2 * i], 0, 0x3120), a0, a1);
                            e4m3_to_h2(__byte_perm(a[2 * i + 1], 0, 0x3120), a2, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma<true>(o[nt][j + i], a0, a1, a2, a3, ph[nt][mt][0], ph[nt][mt][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < JT; ++j) {
                        uint32_t a[4];
                        ldsm_t(a, piece_at(v_at, v_turn, mt * 16, 2 * j));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma<false>(o[nt][j], a[0], a[1], a[2], a[3], ph[nt][mt][0], ph[nt][mt][1]);
                            mma<false>(o[nt][j], a[0], a[1], a[2], a[3], pl[nt][mt][0], pl[nt][mt][1]);
                        }
                    }
                }
            }

            if (kRingLog) {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(empty + stage);
            }
            const bool ended = meta.z & (1 << 31);
            if (ended || it + 1 == tiles) {
                fresh = true;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
                if (began && ended) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float i0 = over<S>(l[nt][0]), i1 = over<S>(l[nt][1]);
                        __nv_bfloat16* const row = static_cast<__nv_bfloat16*>(p.out) + b * p.ldo + static_cast<long long>(head0 + nt * 8) * p.cache.dim;
#pragma unroll
                        for (int j = 0; j < JT; ++j) store_pair<S>(row, p.cache.dim, n_heads - nt * 8, j, lane, o[nt][j], i0, i1);
                        const int h = nt * 8 + 2 * (lane & 3);
                        if (p.lse && lane < 4) {
                            float* lse = p.lse + static_cast<long long>(b) * p.Hq + head0;
                            if (h < n_heads) lse[h] = lse_of<S>(m[nt][0], l[nt][0]);
                            if (h + 1 < n_heads) lse[h + 1] = lse_of<S>(m[nt][1], l[nt][1]);
                        }
                    }
                } else {
                    // what began before this share first, what goes on behind it second
                    // (in the ring, where no more tiles come and its warps are through)
                    const int which = began ? 1 : 0;
                    const bool last = it + 1 == tiles && (!kRingLog || wait_full(empty + stage, parity, p));
                    float* const part = last ? reinterpret_cast<float*>(rings + warp * S::kRing) : p.part + (static_cast<long long>(cta) * S::kWarps + warp) * S::kPart;
                    __syncwarp();
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int j = 0; j < JT; ++j) reinterpret_cast<float4*>(part)[(nt * JT + j) * 32 + lane] = o[nt][j];
                        if (lane < 4) {
                            const int h = nt * 8 + 2 * lane;
                            *reinterpret_cast<float2*>(part + S::kFrag * 4 + h) = make_float2(m[nt][0], m[nt][1]);
                            *reinterpret_cast<float2*>(part + S::kFrag * 4 + S::kHeads + h) = make_float2(l[nt][0], l[nt][1]);
                        }
                    }
                    if (lane == 0) {
                        int f;
                        Open& w = s_open[(beside * turns + turn) * 2 + which];
                        w.first = seg_first;
                        w.end = seg_first + tiles_of<kTile>(p, len, f);
                        w.b = b, w.head0 = head0, w.n_heads = n_heads, w.beside = beside;
                        w.part = part;
                    }
                }
            }
            if (++stage == kRingStages) stage = 0, parity ^= 1;
        }
    }
    __syncthreads();

    // ---------------------------------------------------------------- joins
    // the warps' open slots, a lane each; those of one segment follow one another
    const Open mine = s_open[min(lane, 2 * S::kWarps - 1)];
    const bool any = lane < 2 * S::kWarps && mine.end != 0;
    const uint32_t open = __ballot_sync(0xffffffffu, any), lower = open & ((1u << lane) - 1);
    const int before_me = lower ? 31 - __clz(lower) : 0;
    const int previous = __shfl_sync(0xffffffffu, mine.first, before_me), previous_head = __shfl_sync(0xffffffffu, mine.head0, before_me);
    const bool leads = any && (!lower || previous != mine.first || previous_head != mine.head0);
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    // a segment that this CTA does not have to itself: CTAs c0 .. c1 do.  Of a CTA's
    // two parts of a block of heads the first is of what began before its share or with it.
    const bool shared = leads && (mine.first < cta_from || mine.end > cta_to);
    uint32_t arriving = __ballot_sync(0xffffffffu, shared);
    int c0 = cta, c1 = cta, second = 0;
    if (shared) {
        if (shares.parts) {
            c0 = cta - place, c1 = c0 + shares.parts - 1;
        } else {
            c0 = shares.owner(mine.first), c1 = shares.owner(mine.end - 1);
            second = mine.first != shares.start(c0) ? 1 : 0;       // (of c0)
        }
    }
    const bool grouped = c1 - c0 >= kFlat;
    const int g0 = c0 + (cta - c0) / kGroup * kGroup;          // first CTA of this one's group
    const auto index_of = [&](int c) { return ((2 * c + (c == c0 ? second : 0)) << p.together_log) + mine.beside; };
    float* const cta_parts = p.part + static_cast<long long>(gridDim.x) * S::kWarps * S::kPart;
    float* const group_parts = cta_parts + (static_cast<long long>(gridDim.x) * 2 << p.together_log) * S::kPart;

    // First the CTA's own parts of each segment; then, of segments that CTAs share,
    // the one that arrives last joins theirs.  Many CTAs: the last of each group
    // joins the group's, and the last of those.  (Every warp writes the same lists.)
    uint32_t list = leaders, won = 0;
    for (int round = -1;;) {
        const int count = __popc(list), k = __popc(list & ((1u << lane) - 1));
        const bool in_group = grouped && round == 0, listed = list >> lane & 1;
        if (round < 0) {
            if (any) s_part[__popc(lower)] = mine.part;
            const uint32_t next = leaders & ~((2u << lane) - 1);
            const int n = __popc(next ? open & ((next & -next) - 1) : open) - __popc(lower);
            if (listed) s_joined[k] = {shared ? cta_parts + index_of(cta) * static_cast<long long>(S::kPart) : nullptr, __popc(lower), n, mine.b, mine.head0, mine.n_heads};
        } else {
            const int start = in_group ? g0 : c0, step = grouped && !in_group ? kGroup : 1;
            const int n = in_group ? min(kGroup, c1 + 1 - g0) : (c1 - c0) / step + 1;
            if (listed) s_joined[k] = {in_group ? group_parts + index_of(g0) * static_cast<long long>(S::kPart) : nullptr, k * kFlat, n, mine.b, mine.head0, mine.n_heads};
            for (uint32_t left = list, i = 0; left; left &= left - 1, ++i) {
                const int lead = __ffs(left) - 1;
                const int index0 = __shfl_sync(0xffffffffu, index_of(start), lead), c = __shfl_sync(0xffffffffu, start, lead);
                const int by = __shfl_sync(0xffffffffu, step, lead), parts = __shfl_sync(0xffffffffu, n, lead), beside0 = __shfl_sync(0xffffffffu, mine.beside, lead);
                const int index = lane ? (2 * (c + lane * by) << p.together_log) + beside0 : index0;
                if (lane < parts) s_part[i * kFlat + lane] = (by > 1 ? group_parts : cta_parts) + index * static_cast<long long>(S::kPart);
            }
        }
        __syncwarp();
        // Two column blocks a warp, of wide parts four (where the registers hold them), if
        // half of them each leaves no warp idle: more loads in flight, and the weights
        // worked out once.  Two / one, us: 1 request of 32768, 1 head of 128 for 16, 16.3 /
        // 18.4; 256 up to 2048, 8 for 64, e4m3, 101 / 104.  Four / two: 32 of 2048, 1 head
        // of 256 for 16, e4m3, 22.5 / 24.9.  (Six column blocks: two.)
        constexpr int kBlocks = NT * JT, kLeast = kBlocks > S::kWarps ? 2 : 1, kMost = kLeast == 2 && S::kWarps <= 8 && JT % 4 == 0 ? 4 : 2;
        if (count * kBlocks <= kLeast * S::kWarps) join_all<S, kLeast>(p, s_joined, s_part, count, warp, lane);
        else join_all<S, kMost>(p, s_joined, s_part, count, warp, lane);
        if (round >= 0) arriving |= list & __ballot_sync(0xffffffffu, in_group);
        if (!won) {
            if (!arriving) return;
            ++round;
            __syncthreads();
            if (warp == 0) {
                bool last = false;
                if (arriving >> lane & 1) {
                    const bool of_group = grouped && round == 0;
                    const int all_of = of_group ? min(kGroup, c1 + 1 - g0) : grouped ? (c1 - c0) / kGroup + 1 : c1 - c0 + 1;
                    int* const counter = p.counter + (of_group ? kMaxGrid * 8 + (2 * g0 + (g0 == c0 ? second : 0)) * 8 : c0 * 8) + mine.beside;
                    last = ptx::atom_add_acq_rel_gpu(counter, 1) == all_of - 1;
                    if (last) ptx::st_relaxed_gpu(counter, 0);
                }
                const uint32_t who = __ballot_sync(0xffffffffu, last);
                if (lane == 0) s_won = who;
            }
            arriving = 0;
        }
        __syncthreads();
        if (!won) won = s_won;
        if (!won) return;
        list = 0;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) list |= won & -won, won &= won - 1;
    }
}

// Calls f with the kernel's shape: 16 heads at a time where the group has more
// than 8 (wider heads: their sums do not fit the registers).
template <bool F8, class F>
auto with_shape(int dim, int group, bool pair, F f)
{
    if (dim > 128) {
        if constexpr (!F8)
            if (pair) return dim > 192 ? f(Shape<256, false, 1, true>()) : f(Shape<192, false, 1, true>());
        if constexpr (F8)
            if (group > 8) return dim > 192 ? f(Shape<256, true, 2>()) : f(Shape<192, true, 2>());
        return dim > 192 ? f(Shape<256, F8, 1>()) : f(Shape<192, F8, 1>());
    }
    if (group > 8) return dim > 96 ? f(Shape<128, F8, 2>()) : dim > 64 ? f(Shape<96, F8, 2>()) : f(Shape<64, F8, 2>());
    return dim > 96 ? f(Shape<128, F8, 1>()) : dim > 64 ? f(Shape<96, F8, 1>()) : f(Shape<64, F8, 1>());
}

template <bool F8>
cudaError_t prepare()
{
    const int dims[5] = {64, 96, 128, 192, 256};
    for (int i = 0; i < 15; ++i) {
        const cudaError_t e = with_shape<F8>(dims[i % 5], i < 5 ? 8 : 16, i >= 10, [](auto s) {
            using S = decltype(s);
            return cudaFuncSetAttribute(attn_decode_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        });
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <bool F8>
cudaError_t launch(const AttnParams& p, int num_sms, cudaStream_t stream, bool pdl)
{
    return with_shape<F8>(p.cache.dim, p.group, p.pair, [&](auto s) {
        using S = decltype(s);
        return launch_grid(attn_decode_kernel<S>, p, num_sms, S::kThreads, S::kSmem, stream, false, pdl);
    });
}

}  // namespace attn
}  // namespace tovl
