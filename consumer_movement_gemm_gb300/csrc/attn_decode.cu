// attn_decode.cu -- attention of one new token per request over a paged cache.
//
//   out[b][h] = sum_t softmax_t(scale * q[b][h] . k[t]) v[t]
//
// over the last `window` (or all) of the request's tokens t, whose rows lie in
// the pages of its table.  One pass over the rows: scores, the running maximum
// m, the running sum of exp2(score - m) and the weighted rows of v, rescaled
// where m grows.
//
// The rows are bytes to be streamed, each used for the group's query heads
// only, so the tensor instructions take the rows as their 16-row operand and
// the heads as the 8 columns of the other: S^T = K Q^T and O^T = V^T P^T, with
// S^T's accumulators turned into P^T's fragments by an 8 x 8 transposition in
// registers.  bf16 caches: P enters the second product as two bf16 numbers, its
// upper bits and the rest (2^-15 is left); one bf16 P would add as much error
// as the rounding of the result.  e4m3 caches: rows become fp16 exactly, q fp16
// times a power of two per head, P times the row's scale fp16 (2^-11 of
// itself, below 2^-14 of the largest an absolute 2^-25 of that).
//
// Work: a tile is 16 or 32 rows of one key head for 8 or 16 of its query
// heads.  All tiles of the call, in the order request, head, token, are shared
// out evenly to the warps of a grid that fills the GPU, whatever the lengths.
// A warp streams its tiles through a ring of its own in shared memory
// (cp.async, no CTA barrier), across the ends of segments (one request and
// head).  Segments that several warps share leave (m, sum, O) behind; the CTA
// joins its warps', and of CTAs that share a segment the last to finish joins
// theirs, in the order of the tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "common.cuh"
#include "paged.cuh"
#include "sync.cuh"

namespace tovl {

namespace {

template <int DP_, bool F8_, int NT_>
struct Shape {
    static constexpr int DP = DP_;                 // head dimension, filled up
    static constexpr bool F8 = F8_;
    static constexpr int NT = NT_;                 // blocks of 8 query heads
    static constexpr int kHeads = 8 * NT;
    static constexpr int kRow = DP * (F8 ? 1 : 2);
    static constexpr int kBlockRow = kRow < 128 ? kRow : 128;          // bytes of a row in a column block
    static constexpr int CB = kRow / kBlockRow;
    static constexpr int kTile = kRow <= 64 ? 64 : kRow <= 128 ? 32 : 16;
    static constexpr int kBlock = kTile * kBlockRow;
    static constexpr int kRows = CB * kBlock;      // all of k or of v
    static constexpr int MT = kTile / 16;
    static constexpr int JT = DP / 16;             // blocks of 16 columns
    static constexpr int kStage = 2 * kRows;
    static constexpr int kScaleStage = F8 ? 2 * kTile * 4 : 0;
    static constexpr int kWarps = kRow > 256 ? 6 : NT == 1 ? 12 : 8;
    static constexpr int kFit = (222 * 1024) / (kWarps * (kStage + kScaleStage));
    static constexpr int kStages = kFit > 4 ? 4 : kFit;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kScales = kStages * kScaleStage;               // of a warp, behind all rings
    static constexpr int kSmem = kWarps * (kRing + kScales) + 1024;
    static constexpr int kFrag = NT * JT * 32;     // float4 of one O
    static constexpr int kPart = kFrag * 4 + 2 * kHeads;               // floats of a part: O, m, sum
    // the 16-byte pieces of row r of a block are exchanged by XOR with this
    // (so that 8 rows' pieces lie in different banks; the copies' swizzle)
    static __host__ __device__ constexpr int phase(int r) { return kBlockRow == 128 ? r & 7 : (r >> 1) & 3; }
    static_assert(kBlockRow == 64 || kBlockRow == 128, "swizzle");
    static_assert(kStages >= 2 && kBlock % 1024 == 0 && kPart * 4 <= kRing, "ring");
};

// What is left behind of a segment that does not lie within one warp's share.
struct Open {
    long long first, end;      // its tiles in the order of the call; end == 0: none
    const float* part;
    int b, head0, n_heads;     // its request and query heads
    int beside;                // which of the heads that go together
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
// two e4m3 numbers (exactly)
__device__ __forceinline__ uint32_t e4m3_to_h2(uint32_t two)
{
    uint32_t d;
    asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(d) : "r"(two));
    return d;
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// What the upper half of a weight's bits leaves.  It has the weight's sign even
// where nothing is left, so that both products with an infinite value have too.
__device__ __forceinline__ float rest(float w) { return fmaxf(w - bf_hi(__float_as_uint(w)), w * 0x1p-30f); }

// The weight of e4m3 rows is exp2(score - m) times the row's scale, m the
// largest score + log2(scale), so that the product's operand is 1 at most.  The
// sum takes the same exponential without the scale; the shift keeps it inside
// fp32 for any scale that a row of finite bf16 numbers can have (2^-49 .. 2^120).
constexpr float kShift = 40.f;

// First tile and number of tiles of a request.
template <int TILE>
__device__ __forceinline__ int tiles_of(const AttnParams& p, int len, int& first)
{
    const int lo = p.window && len > p.window ? len - p.window : 0;
    first = lo / TILE;
    return len > 0 ? (len - 1) / TILE + 1 - first : 0;
}

__device__ __forceinline__ int length_of(const AttnParams& p, int b)
{
    const int len = __ldg(p.length + b);
    const long long most = static_cast<long long>(p.width) * p.cache.page;
    return len < 0 ? 0 : len > most ? static_cast<int>(most) : len;
}

// A place in the order of the call: request, key head, block of its query
// heads, tile.
template <class S>
struct Cursor {
    long long left;            // tiles of the share from here on
    long long at;              // linear tile
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
        head = per_head == 1 ? v : v / per_head;
        block = v - head * per_head;
    }
    // together: blocks of heads that neighbouring warps take side by side
    __device__ __forceinline__ void next(const AttnParams& p, int per_head, int together)
    {
        --left;
        ++at;
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

// What a sum of weights divides: 1 / l, without the shift.
template <class S>
__device__ __forceinline__ float over(float l)
{
    return l == 0.f ? 0.f : __fdividef(S::F8 ? 0x1p40f : 1.f, l);
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

// Element e of the joined parts of one segment, with the statistics of its two
// heads, in the order of the parts; four are in flight at a time.
template <class S, bool FAR, class Part>
__device__ __forceinline__ float4 join(int count, Part part, int e, int h, float2& m, float2& l)
{
    constexpr int kAhead = 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    m = make_float2(-INFINITY, -INFINITY), l = make_float2(0.f, 0.f);
    for (int i = 0; i < count; i += kAhead) {
        float2 pm[kAhead], pl[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            pm[k] = make_float2(-INFINITY, -INFINITY), pl[k] = make_float2(0.f, 0.f), v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i + k >= count) continue;
            const float* q = part(i + k);
            const float2* stats = reinterpret_cast<const float2*>(q + S::kFrag * 4 + h);
            if (FAR) {
                pm[k] = __ldcg(stats), pl[k] = __ldcg(stats + S::kHeads / 2), v[k] = __ldcg(reinterpret_cast<const float4*>(q) + e);
            } else {
                pm[k] = *stats, pl[k] = stats[S::kHeads / 2], v[k] = reinterpret_cast<const float4*>(q)[e];
            }
        }
        float2 top = m;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) top.x = fmaxf(top.x, pm[k].x), top.y = fmaxf(top.y, pm[k].y);
        const float u0 = top.x == -INFINITY ? 0.f : top.x, u1 = top.y == -INFINITY ? 0.f : top.y;
        const float c0 = ex2(m.x - u0), c1 = ex2(m.y - u1);
        o.x *= c0, o.y *= c1, o.z *= c0, o.w *= c1, l.x *= c0, l.y *= c1;
        m = top;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float w0 = ex2(pm[k].x - u0), w1 = ex2(pm[k].y - u1);
            o.x += v[k].x * w0, o.y += v[k].y * w1, o.z += v[k].z * w0, o.w += v[k].w * w1;
            l.x += pl[k].x * w0, l.y += pl[k].y * w1;
        }
    }
    return o;
}

// Tiles that a warp gets before more CTAs share a segment.
constexpr int kLeast = 3;

// CTAs that share a segment join in groups where there are more than kFlat.
constexpr int kFlat = 24;
constexpr int kGroup = 12;

// n i / turns, i <= turns <= 8
__device__ __forceinline__ long long part_of(long long n, int turns, int i)
{
    if (n < (1 << 28)) return static_cast<unsigned>(n) * i / static_cast<unsigned>(turns);
    return n * i / turns;
}

// First tile of CTA c's share, and the CTA of a tile.
__device__ __forceinline__ long long share_of(long long total, int ctas, int c)
{
    if (total < (1 << 24)) return static_cast<unsigned>(total) * c / ctas;
    return total * c / ctas;
}
__device__ __forceinline__ int cta_of(long long total, int ctas, long long tile)
{
    if (total < (1 << 24)) return (static_cast<unsigned>(tile + 1) * ctas - 1) / static_cast<unsigned>(total);
    return static_cast<int>(((tile + 1) * ctas - 1) / total);
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1) attn_decode_kernel(const __grid_constant__ AttnParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_full[S::kWarps][S::kStages];
    __shared__ int4 s_meta[S::kWarps][S::kStages];
    __shared__ long long s_sum[S::kWarps];
    __shared__ int s_flags[S::kWarps];
    __shared__ long long s_before[S::kThreads];
    __shared__ Open s_open[S::kWarps * 2];
    __shared__ uint32_t s_won;
    constexpr int kTile = S::kTile, NT = S::NT, JT = S::JT, MT = S::MT, kStages = S::kStages, CB = S::CB;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        ptx::prefetch_tmap(&p.k_map);
        ptx::prefetch_tmap(&p.v_map);
    }
    if (lane < kStages) ptx::mbar_init(&s_full[warp][lane], 1);
    if (lane < 2) s_open[warp * 2 + lane].end = 0;
    ptx::fence_mbar_init();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    // ---------------------------------------------------------------- shares
    const int per_head = (p.group + S::kHeads - 1) / S::kHeads, together = 1 << p.together_log;
    const int groups = p.cache.heads * per_head >> p.together_log;
    const int beside = warp & (together - 1), turn = warp >> p.together_log, turns = S::kWarps >> p.together_log;
    const int chunk = (p.B + S::kThreads - 1) / S::kThreads, b0 = tid * chunk;
    long long sum = 0;
    bool none = false, equal = true;
    int first_count, unused;
    first_count = tiles_of<kTile>(p, length_of(p, 0), unused);
    for (int b = b0; b < min(p.B, b0 + chunk); ++b) {
        const int len = __ldg(p.length + b);
        if (len < 0 || len > static_cast<long long>(p.width) * p.cache.page) record_error(p.ctrl, kErrInvalid);
        const int count = tiles_of<kTile>(p, length_of(p, b), unused);
        sum += count;
        none |= len <= 0;
        equal &= count == first_count;
    }
    long long before = sum;                  // inclusive prefix
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    if (lane == 31) s_sum[warp] = before;
    none = __any_sync(0xffffffffu, none), equal = __all_sync(0xffffffffu, equal);
    if (lane == 31) s_flags[warp] = (none ? 1 : 0) | (equal ? 0 : 2);
    __syncthreads();
    int flags = 0;
    long long total = 0;
#pragma unroll
    for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
        flags |= s_flags[w];
    }
    before = (before - sum) * groups;
    total *= groups;
    // CTAs that get work: all, or so many that a warp has kLeast tiles; with segments
    // of one length a multiple of them, so that few CTAs (or one) share a segment
    const int cta = blockIdx.x;
    int ctas = gridDim.x;
    if (total < static_cast<long long>(gridDim.x) * turns * kLeast) {
        const int segments = p.B * groups, per_segment = (first_count + turns * kLeast - 1) / (turns * kLeast);
        const bool even = !(flags & 2) && static_cast<long long>(segments) * per_segment <= static_cast<int>(gridDim.x);
        ctas = even ? segments * per_segment : (static_cast<int>(total) + turns * kLeast - 1) / (turns * kLeast);
    }
    // requests without tokens: nothing of theirs is in the order
    for (int b = blockIdx.x; (flags & 1) && b < p.B; b += gridDim.x) {
        if (__ldg(p.length + b) > 0) continue;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + b * p.ldo;
        for (int i = tid; i < p.Hq * p.cache.dim; i += S::kThreads) out[i] = __float2bfloat16(0.f);
        if (p.lse)
            for (int i = tid; i < p.Hq; i += S::kThreads) p.lse[static_cast<long long>(b) * p.Hq + i] = -INFINITY;
    }
    if (cta >= ctas) return;
    const long long cta_from = share_of(total, ctas, cta), cta_to = share_of(total, ctas, cta + 1);
    s_before[tid] = before;
    __syncthreads();

    // this warp's share: the last thread's requests that begin at its first tile or before
    Cursor<S> put;
    {
        const long long share = cta_to - cta_from, from = cta_from + part_of(share, turns, turn);
        put.left = cta_from + part_of(share, turns, turn + 1) - from;
        put.at = from;
        constexpr int kPer = S::kThreads / 32;
        const int coarse = __popc(__ballot_sync(0xffffffffu, s_before[lane * kPer] <= from)) - 1;
        const int at = coarse * kPer + __popc(__ballot_sync(0xffffffffu, lane < kPer && s_before[coarse * kPer + min(lane, kPer - 1)] <= from)) - 1;
        long long r = from - s_before[at];
        for (put.b = at * chunk;; ++put.b) {
            put.enter(p);
            if (r < static_cast<long long>(put.count) * groups) break;
            r -= static_cast<long long>(put.count) * groups;
        }
        const int group = r < (1LL << 31) ? static_cast<int>(static_cast<unsigned>(r) / static_cast<unsigned>(put.count)) : static_cast<int>(r / put.count);
        put.at_head(group * together + beside, per_head);
        put.tile = put.first + static_cast<int>(r - static_cast<long long>(group) * put.count);
    }

    // ---------------------------------------------------------------- a warp's stream
    uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023)) + warp * S::kRing;
    uint8_t* const ring_scales = ring + (S::kWarps - warp) * S::kRing + warp * S::kScales;
    const uint32_t ring_u = ptx::smem_u32(ring), scales_u = ptx::smem_u32(ring_scales);
    const long long tiles = put.left, warp_from = put.at;
    const auto page_of = [&](int t) {
        return p.cache.page_shift >= 0 ? t >> p.cache.page_shift : static_cast<int>(static_cast<unsigned>(t) / static_cast<unsigned>(p.cache.page));
    };
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
                const int n = page_of(t);
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
                s_meta[warp][stage] = make_int4(put.b, put.head | put.block << 16, put.tile | (put.tile == put.first ? 1 << 30 : 0) | (put.tile == last ? 1 << 31 : 0), put.len);
            }
            if (page_id[0] == -2 || page_id[kOwn - 1] == -2) record_error(p.ctrl, kErrInvalid);
            if (p.boxed) {
                // what holds no token of this tile is outside the tensor: zeros, and nothing read
                uint64_t* const full = &s_full[warp][stage];
                const uint32_t bar = ptx::smem_u32(full);
                const bool in = page_id[0] >= 0;
                uint32_t bytes = 2 * S::kRows;
                if (S::F8) bytes += 8 * box_rows * __popc(__ballot_sync(0xffffffffu, in && lane < 1 << pieces_log));
                if (lane == 0) ptx::mbar_arrive_expect_tx(full, bytes);
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
                    const int row = i * 32 / kPerRow + lane / kPerRow, c = lane % kPerRow;
                    static_assert(kPerRow <= 32, "a row is one instruction's at most");
                    const long long o = __shfl_sync(0xffffffffu, off[i * 32 / kPerRow / 32], row & 31);
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
        find_pages();
#pragma unroll 1
        for (int s = 0; s < kStages - 1; ++s) fetch(s);
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
        long long seg_first = 0;
        bool began = false, fresh = true;
        int stage = 0;
        uint32_t parity = 0;
        for (long long it = 0; it < tiles; ++it) {
            __syncwarp();
            const int4 meta = s_meta[warp][stage];
            const int b = meta.x, tile = meta.z & 0x3fffffff, len = meta.w;
            const int block = meta.y >> 16, head0 = (meta.y & 0xffff) * p.group + block * S::kHeads, n_heads = min(S::kHeads, p.group - block * S::kHeads);
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
                    const int h = nt * 8 + (lane >> 2);
                    const __nv_bfloat16* row = qp + static_cast<long long>(head0 + h) * p.cache.dim;
                    float top = 0.f;
#pragma unroll
                    for (int j = 0; j < JT; ++j) {
                        if constexpr (S::F8) {
                            const int d = 16 * j + 4 * (lane & 3);
                            const uint2 u = h < n_heads && d < p.cache.dim ? __ldg(reinterpret_cast<const uint2*>(row + d)) : make_uint2(0, 0);
                            q[nt][j][0] = u.x, q[nt][j][1] = u.y;
                            top = fmaxf(top, fmaxf(fmaxf(fabsf(bf_lo(u.x)), fabsf(bf_hi(u.x))), fmaxf(fabsf(bf_lo(u.y)), fabsf(bf_hi(u.y)))));
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int d = 16 * j + 8 * i + 2 * (lane & 3);
                                q[nt][j][i] = h < n_heads && d < p.cache.dim ? __ldg(reinterpret_cast<const uint32_t*>(row + d)) : 0u;
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
            if (p.boxed) {
                if (!wait_full(&s_full[warp][stage], parity, p)) {
                    // the other copies in flight, then out
                    for (int s = 1; s < kStages - 1 && it + s < tiles; ++s) {
                        if (++stage == kStages) stage = 0, parity ^= 1;
                        wait_full(&s_full[warp][stage], parity, p);
                    }
                    break;
                }
            } else {
                cp_wait<kStages - 2>();
            }
            __syncwarp();
            fetch(stage == 0 ? kStages - 1 : stage - 1);
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
                            const uint32_t r0 = a[2 * i], r1 = a[2 * i + 1];
                            const uint32_t a0 = e4m3_to_h2(r0 & 0xffff), a2 = e4m3_to_h2(r0 >> 16), a1 = e4m3_to_h2(r1 & 0xffff), a3 = e4m3_to_h2(r1 >> 16);
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
                        vl[mt][i] = fmaxf(lg2(scales[kTile + r]), -80.f);
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
            uint32_t ph[NT][MT][2], pl[NT][MT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    m0 = fmaxf(m0, fmaxf(s[nt][mt].x + vl[mt][0], s[nt][mt].z + vl[mt][1]));
                    m1 = fmaxf(m1, fmaxf(s[nt][mt].y + vl[mt][0], s[nt][mt].w + vl[mt][1]));
                }
#pragma unroll
                for (int d = 4; d < 32; d *= 2) {
                    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
                    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
                }
                m0 = fmaxf(m0, m[nt][0]), m1 = fmaxf(m1, m[nt][1]);
                // (all scores -inf so far: weights of 0)
                const float u0 = (m0 == -INFINITY ? 0.f : m0) - (S::F8 ? kShift : 0.f), u1 = (m1 == -INFINITY ? 0.f : m1) - (S::F8 ? kShift : 0.f);
                if (__any_sync(0xffffffffu, m0 != m[nt][0] || m1 != m[nt][1])) {
                    const float c0 = m[nt][0] == -INFINITY ? 0.f : ex2(m[nt][0] - m0), c1 = m[nt][1] == -INFINITY ? 0.f : ex2(m[nt][1] - m1);
                    l[nt][0] *= c0, l[nt][1] *= c1;
#pragma unroll
                    for (int j = 0; j < JT; ++j) o[nt][j].x *= c0, o[nt][j].y *= c1, o[nt][j].z *= c0, o[nt][j].w *= c1;
                    m[nt][0] = m0, m[nt][1] = m1;
                }
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
                            const uint32_t r0 = __byte_perm(a[2 * i], 0, 0x3120), r1 = __byte_perm(a[2 * i + 1], 0, 0x3120);
                            const uint32_t a0 = e4m3_to_h2(r0 & 0xffff), a1 = e4m3_to_h2(r0 >> 16), a2 = e4m3_to_h2(r1 & 0xffff), a3 = e4m3_to_h2(r1 >> 16);
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
                    // (in the ring, where no more tiles come)
                    const int which = began ? 1 : 0;
                    float* const part = it + 1 == tiles ? reinterpret_cast<float*>(ring) : p.part + (static_cast<long long>(cta) * S::kWarps + warp) * S::kPart;
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
            if (++stage == kStages) stage = 0, parity ^= 1;
        }
    }
    __syncthreads();

    // ---------------------------------------------------------------- joins
    // the warps' open slots, a lane each; those of one segment follow one another
    const Open mine = s_open[min(lane, 2 * S::kWarps - 1)];
    const bool any = lane < 2 * S::kWarps && mine.end != 0;
    const uint32_t open = __ballot_sync(0xffffffffu, any), lower = open & ((1u << lane) - 1);
    const int before_me = lower ? 31 - __clz(lower) : 0;
    const long long previous = __shfl_sync(0xffffffffu, mine.first, before_me);
    const int previous_head = __shfl_sync(0xffffffffu, mine.head0, before_me);
    const bool leads = any && (!lower || previous != mine.first || previous_head != mine.head0);
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    // a segment that this CTA does not have to itself: CTAs c0 .. c1 do.  Of a CTA's
    // two parts of a block of heads the first is of what began before its share or with it.
    const bool shares = leads && (mine.first < cta_from || mine.end > cta_to);
    const uint32_t shared = __ballot_sync(0xffffffffu, shares);
    int c0 = cta, c1 = cta, second = 0;
    if (shares) {
        c0 = cta_of(total, ctas, mine.first), c1 = cta_of(total, ctas, mine.end - 1);
        second = mine.first != share_of(total, ctas, c0) ? 1 : 0;      // (of c0)
    }
    const int g0 = c0 + (cta - c0) / kGroup * kGroup;       // first CTA of this one's group
    const auto index_of = [&](int c, int from, int sec, int which) { return ((2 * c + (c == from ? sec : 0)) << p.together_log) + which; };
    float* const cta_parts = p.part + static_cast<long long>(gridDim.x) * S::kWarps * S::kPart;
    float* const group_parts = cta_parts + (static_cast<long long>(gridDim.x) * 2 << p.together_log) * S::kPart;

    // what a thread does with its share of a segment's join; to: where a joined part
    // goes, null: it is the result
    const auto put_joined = [&](const Open& seg, float* to, int e, float4 o, float2 m, float2 l) {
        const int ln = e & 31, j = e / 32 % JT, nt = e / 32 / JT, h = nt * 8 + 2 * (ln & 3);
        const bool stats = j == 0 && ln < 4;
        if (to) {
            reinterpret_cast<float4*>(to)[e] = o;
            if (stats) {
                *reinterpret_cast<float2*>(to + S::kFrag * 4 + h) = m;
                *reinterpret_cast<float2*>(to + S::kFrag * 4 + S::kHeads + h) = l;
            }
            return;
        }
        const int head0 = seg.head0, n_heads = seg.n_heads;
        store_pair<S>(static_cast<__nv_bfloat16*>(p.out) + seg.b * p.ldo + static_cast<long long>(head0 + nt * 8) * p.cache.dim, p.cache.dim,
                      n_heads - nt * 8, j, ln, o, over<S>(l.x), over<S>(l.y));
        if (stats && p.lse) {
            float* lse = p.lse + static_cast<long long>(seg.b) * p.Hq + head0;
            if (h < n_heads) lse[h] = lse_of<S>(m.x, l.x);
            if (h + 1 < n_heads) lse[h + 1] = lse_of<S>(m.y, l.y);
        }
    };
    const auto head_of = [](int e) { return e / 32 / JT * 8 + 2 * (e & 3); };
    // f(slot, first element, step) for the slots of a mask, shared out to the warps
    const auto each = [&](uint32_t slots, auto f) {
        if (!slots) return;
        const int count = __popc(slots), teams = min(count, S::kWarps), team = warp % teams, mates = (S::kWarps - team + teams - 1) / teams;
        for (int k = 0; slots; ++k, slots &= slots - 1)
            if (k % teams == team) f(__ffs(slots) - 1, warp / teams * 32 + lane, mates * 32);
    };
    // this CTA's parts of each segment
    each(leaders, [&](int lead, int first, int step) {
        const uint32_t next = leaders & ~((2u << lead) - 1);
        const uint32_t slots = open & ~((1u << lead) - 1) & (next ? (next & -next) - 1 : 0xffffffffu);
        const int index = __shfl_sync(0xffffffffu, index_of(cta, c0, second, mine.beside), lead);
        float* const to = shared >> lead & 1 ? cta_parts + index * static_cast<long long>(S::kPart) : nullptr;
        for (int e = first; e < S::kFrag; e += step) {
            float2 m, l;
            uint32_t left = slots;
            const float4 o = join<S, false>(__popc(slots), [&](int) {
                const float* part = s_open[__ffs(left) - 1].part;
                left &= left - 1;
                return part;
            }, e, head_of(e), m, l);
            put_joined(s_open[lead], to, e, o, m, l);
        }
    });
    if (!shared) return;
    // few CTAs: the last joins all; many: the last of each group does, and the last of those
    const bool grouped = c1 - c0 >= kFlat;
    uint32_t arriving = shared;
#pragma unroll 1
    for (int round = 0; arriving; ++round) {
        __syncthreads();
        const bool in_group = grouped && round == 0;
        if (warp == 0) {
            bool last = false;
            if (arriving >> lane & 1) {
                const int count = in_group ? min(kGroup, c1 + 1 - g0) : grouped ? (c1 - c0) / kGroup + 1 : c1 - c0 + 1;
                int* const counter = p.counter + (in_group ? kMaxGrid * 8 + (2 * g0 + (g0 == c0 ? second : 0)) * 8 : c0 * 8) + mine.beside;
                last = ptx::atom_add_acq_rel_gpu(counter, 1) == count - 1;
                if (last) ptx::st_relaxed_gpu(counter, 0);
            }
            const uint32_t won = __ballot_sync(0xffffffffu, last);
            if (lane == 0) s_won = won;
        }
        __syncthreads();
        const uint32_t won = s_won;
        each(won, [&](int lead, int first, int step) {
            const bool group = __shfl_sync(0xffffffffu, in_group, lead), of_groups = __shfl_sync(0xffffffffu, grouped, lead) && !group;
            const int from = __shfl_sync(0xffffffffu, c0, lead), sec = __shfl_sync(0xffffffffu, second, lead), which = __shfl_sync(0xffffffffu, mine.beside, lead);
            const int start = group ? __shfl_sync(0xffffffffu, g0, lead) : from, to_cta = __shfl_sync(0xffffffffu, c1, lead);
            const int count = group ? min(kGroup, to_cta + 1 - start) : of_groups ? (to_cta - from) / kGroup + 1 : to_cta - from + 1;
            const float* const base = of_groups ? group_parts : cta_parts;
            const int stride = of_groups ? kGroup : 1;
            const auto part = [&](int k) { return base + index_of(start + k * stride, from, sec, which) * static_cast<long long>(S::kPart); };
            float* const to = group ? group_parts + index_of(start, from, sec, which) * static_cast<long long>(S::kPart) : nullptr;
            for (int e = first; e < S::kFrag; e += step) {
                float2 m, l;
                const float4 o = join<S, true>(count, part, e, head_of(e), m, l);
                put_joined(s_open[lead], to, e, o, m, l);
            }
        });
        arriving = won & __ballot_sync(0xffffffffu, in_group);
    }
}

template <class S>
cudaError_t launch(const AttnParams& p, int num_sms, cudaStream_t stream, bool pdl)
{
    return launch_grid(attn_decode_kernel<S>, p, num_sms, S::kThreads, S::kSmem, stream, false, pdl);
}

// Calls f with the kernel's shape: 16 heads at a time where the group has more
// than 8 (256 columns: their sums do not fit the registers).
template <class F>
auto with_shape(int dim, bool e4m3, int group, F f)
{
    if (dim > 128) return e4m3 ? f(Shape<256, true, 1>()) : f(Shape<256, false, 1>());
    if (dim > 64) {
        if (group > 8) return e4m3 ? f(Shape<128, true, 2>()) : f(Shape<128, false, 2>());
        return e4m3 ? f(Shape<128, true, 1>()) : f(Shape<128, false, 1>());
    }
    if (group > 8) return e4m3 ? f(Shape<64, true, 2>()) : f(Shape<64, false, 2>());
    return e4m3 ? f(Shape<64, true, 1>()) : f(Shape<64, false, 1>());
}

template <class S>
long long parts_bytes(int num_sms, int together)
{
    return 4LL * S::kPart * num_sms * (S::kWarps + 4 * together);
}

}  // namespace

AttnShape attn_decode_shape(int dim, bool e4m3, int group)
{
    return with_shape(dim, e4m3, group, [&](auto s) {
        using S = decltype(s);
        return AttnShape{S::kTile, S::kBlockRow, S::kWarps, S::kHeads};
    });
}

int attn_decode_together(const AttnShape& s, int heads, int dim, bool e4m3, int group)
{
    const int blocks = (group + s.heads - 1) / s.heads, row = dim * (e4m3 ? 1 : 2);
    int n = 1;
    while (blocks == 1 && n < 8 && n * row % 128 && heads % (2 * n) == 0 && s.warps % (2 * n) == 0) n *= 2;
    return n;
}

long long attn_decode_workspace(int heads, int group, int dim, int num_sms)
{
    long long most = 0;
    for (int e4m3 = 0; e4m3 < 2; ++e4m3) {
        const AttnShape shape = attn_decode_shape(dim, e4m3, group);
        const int together = attn_decode_together(shape, heads, dim, e4m3, group);
        const long long bytes = with_shape(dim, e4m3, group, [&](auto s) { return parts_bytes<decltype(s)>(num_sms, together); });
        if (bytes > most) most = bytes;
    }
    return most;
}

cudaError_t prepare_attn_decode()
{
    const int dims[3] = {64, 128, 256};
    for (int i = 0; i < 12; ++i) {
        const cudaError_t e = with_shape(dims[i / 4], i & 1, i & 2 ? 16 : 8, [](auto s) {
            using S = decltype(s);
            return cudaFuncSetAttribute(attn_decode_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        });
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_attn_decode(const AttnParams& p, bool e4m3, int num_sms, cudaStream_t stream, bool pdl)
{
    return with_shape(p.cache.dim, e4m3, p.group, [&](auto s) { return launch<decltype(s)>(p, num_sms, stream, pdl); });
}

}  // namespace tovl
