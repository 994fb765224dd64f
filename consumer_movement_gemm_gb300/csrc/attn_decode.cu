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
    static constexpr int kPitch = kRow + 16;       // rows start 4 banks apart
    static constexpr int kTile = kRow <= 128 ? 32 : 16;
    static constexpr int MT = kTile / 16;
    static constexpr int JT = DP / 16;             // blocks of 16 columns
    static constexpr int kScales = 2 * kTile * kPitch;                 // offset in a stage
    static constexpr int kMeta = kScales + (F8 ? 2 * kTile * 4 : 0);
    static constexpr int kStage = kMeta + 16;
    static constexpr int kWarps = kStage > 16000 ? 4 : 8;
    static constexpr int kFit = (224 * 1024) / (kWarps * kStage);
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kSmem = kWarps * kStages * kStage;
    static constexpr int kFrag = NT * JT * 32;     // float4 of one O
    static constexpr int kPart = kFrag * 4 + 2 * kHeads;               // floats of a part: O, m, sum
    static_assert(kStages >= 3, "ring");
};

// What is left behind of a segment that does not lie within one warp's share.
struct Open {
    long long first, end;      // its tiles in the order of the call
    int b, vh;                 // end == 0: none
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

// A place in the order of the call: request, block of heads, tile.
template <class S>
struct Cursor {
    long long left;            // tiles of the share from here on
    long long at;              // linear tile
    int b, vh, tile;
    int len, first, count;     // of the request

    __device__ __forceinline__ void enter(const AttnParams& p)
    {
        len = length_of(p, b);
        count = tiles_of<S::kTile>(p, len, first);
    }
    __device__ __forceinline__ void next(const AttnParams& p, int heads)
    {
        --left;
        ++at;
        if (++tile < first + count || left == 0) return;
        if (++vh == heads) {
            vh = 0;
            do {
                ++b;
                enter(p);
            } while (count == 0);       // (a share ends at the last request with tiles)
        }
        tile = first;
    }
};

// What a sum of weights divides: 1 / l, without the shift.
template <class S>
__device__ __forceinline__ float over(float l)
{
    return l == 0.f ? 0.f : (S::F8 ? 0x1p40f : 1.f) / l;
}

// Column c (0 .. 3 of a float4) of the fragment block j of lane `lane` is
// element dim_of(), head 2 (lane % 4) + (c & 1).
template <bool F8>
__device__ __forceinline__ int dim_of(int j, int lane, int c)
{
    const int g = lane >> 2;
    return 16 * j + (F8 ? 2 * g + (c >> 1) : g + 8 * (c >> 1));
}

// out and lse of one float4 of a segment's result
template <class S>
__device__ __forceinline__ void store_one(const AttnParams& p, int b, int head0, int heads, int j, int lane, float4 o)
{
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + b * p.ldo;
    const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int d = dim_of<S::F8>(j, lane, c), h = 2 * (lane & 3) + (c & 1);
        if (h < heads && d < p.cache.dim) out[static_cast<long long>(head0 + h) * p.cache.dim + d] = __float2bfloat16(v[c]);
    }
}

template <class S>
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l > 0.f || l != l ? (m + log2f(l) - (S::F8 ? kShift : 0.f)) * 0.693147180559945309f : -INFINITY;
}

// Joins `count` parts (part(i): its floats) of one segment; f gets each float4
// and where it belongs, g the statistics.  All threads of the CTA.
template <class S, class Part, class F, class G>
__device__ __forceinline__ void join(int count, Part part, F f, G g)
{
    for (int e = threadIdx.x; e < S::kFrag; e += S::kThreads) {
        const int lane = e & 31, j = e / 32 % S::JT, nt = e / 32 / S::JT;
        const int h = nt * 8 + 2 * (lane & 3);
        float m0 = -INFINITY, m1 = -INFINITY;
        for (int i = 0; i < count; ++i) {
            const float2 m = __ldcg(reinterpret_cast<const float2*>(part(i) + S::kFrag * 4 + h));
            m0 = fmaxf(m0, m.x), m1 = fmaxf(m1, m.y);
        }
        const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float l0 = 0.f, l1 = 0.f;
        for (int i = 0; i < count; ++i) {
            const float* q = part(i);
            const float2 m = __ldcg(reinterpret_cast<const float2*>(q + S::kFrag * 4 + h));
            const float2 l = __ldcg(reinterpret_cast<const float2*>(q + S::kFrag * 4 + S::kHeads + h));
            const float4 v = __ldcg(reinterpret_cast<const float4*>(q) + e);
            const float w0 = ex2(m.x - u0), w1 = ex2(m.y - u1);
            o.x += v.x * w0, o.y += v.y * w1, o.z += v.z * w0, o.w += v.w * w1;
            l0 += l.x * w0, l1 += l.y * w1;
        }
        f(e, nt, j, lane, o, l0, l1);
        if (j == 0 && lane < 4) g(h, m0, m1, l0, l1);
    }
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1) attn_decode_kernel(const AttnParams p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_sum[S::kWarps];
    __shared__ Cursor<S> s_start[S::kWarps];
    __shared__ Open s_open[S::kWarps * 2];
    __shared__ int s_last;
    constexpr int kTile = S::kTile, NT = S::NT, JT = S::JT, MT = S::MT, kStages = S::kStages;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    // ---------------------------------------------------------------- shares
    const int per_head = (p.group + S::kHeads - 1) / S::kHeads, heads = p.cache.heads * per_head;
    const int chunk = (p.B + S::kThreads - 1) / S::kThreads, b0 = tid * chunk;
    long long sum = 0;
    for (int b = b0; b < min(p.B, b0 + chunk); ++b) {
        const int len = __ldg(p.length + b);
        int first;
        if (len < 0 || len > static_cast<long long>(p.width) * p.cache.page) record_error(p.ctrl, kErrInvalid);
        sum += tiles_of<kTile>(p, length_of(p, b), first);
    }
    long long before = sum;                  // inclusive prefix
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    if (lane == 31) s_sum[warp] = before;
    if (lane < 2) s_open[warp * 2 + lane].end = 0;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    before -= sum;
    total *= heads;
    // CTAs that get work: as many as the warps' tiles need, or all
    const long long want = (total + S::kWarps - 1) / S::kWarps;
    const int ctas = static_cast<int>(want < gridDim.x ? want : gridDim.x), warps = ctas * S::kWarps;
    const int cta = blockIdx.x;
    // requests without tokens: nothing of theirs is in the order
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (__ldg(p.length + b) > 0) continue;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + b * p.ldo;
        for (int i = tid; i < p.Hq * p.cache.dim; i += S::kThreads) out[i] = __float2bfloat16(0.f);
        if (p.lse)
            for (int i = tid; i < p.Hq; i += S::kThreads) p.lse[static_cast<long long>(b) * p.Hq + i] = -INFINITY;
    }
    if (cta >= ctas) return;
    for (int w = 0; w < S::kWarps; ++w) {
        const long long from = (static_cast<long long>(cta) * S::kWarps + w) * total / warps;
        const long long to = (static_cast<long long>(cta) * S::kWarps + w + 1) * total / warps;
        if (from < before * heads || from >= (before + sum) * heads) continue;
        Cursor<S> c;
        c.left = to - from;
        c.at = from;
        long long r = from - before * heads;
        for (c.b = b0;; ++c.b) {
            c.enter(p);
            if (r < static_cast<long long>(c.count) * heads) break;
            r -= static_cast<long long>(c.count) * heads;
        }
        c.vh = static_cast<int>(r / c.count);
        c.tile = c.first + static_cast<int>(r % c.count);
        s_start[w] = c;
    }
    __syncthreads();

    // ---------------------------------------------------------------- a warp's stream
    float* const scratch = p.part + (static_cast<long long>(cta) * S::kWarps + warp) * 2 * S::kPart;
    uint8_t* const ring = smem + warp * kStages * S::kStage;
    const uint32_t ring_u = ptx::smem_u32(ring);
    Cursor<S> put = s_start[warp];
    const long long tiles = put.left;
    int page_id = -1;
    const auto find_page = [&]() {
        const int t = put.tile * kTile + lane;
        const int lo = p.window && put.len > p.window ? put.len - p.window : 0;
        page_id = -1;
        if (put.left > 0 && lane < kTile && t >= lo && t < put.len) {
            const int slot = p.cache.page_shift >= 0 ? t >> p.cache.page_shift : static_cast<int>(static_cast<unsigned>(t) / static_cast<unsigned>(p.cache.page));
            page_id = __ldg(p.table + put.b * p.ldt + slot);
            if (static_cast<unsigned>(page_id) >= static_cast<unsigned>(p.cache.pages)) page_id = -2;
        }
    };
    // starts the copies of the tile at `put` and moves on
    const auto fetch = [&](int stage) {
        if (put.left > 0) {
            const uint32_t dst = ring_u + stage * S::kStage;
            const int t = put.tile * kTile + lane, head = put.vh / per_head;
            long long off = -1;
            if (page_id >= 0) {
                const int in = p.cache.page_shift >= 0 ? t & (p.cache.page - 1) : static_cast<int>(static_cast<unsigned>(t) % static_cast<unsigned>(p.cache.page));
                off = page_id * p.cache.page_stride + in * p.cache.slot_stride + head * p.cache.head_stride;
                if (S::F8) {
                    const long long at = (static_cast<long long>(page_id) * p.cache.heads + head) * p.cache.page + in;
                    cp_async4(dst + S::kScales + lane * 4, p.cache.k_scale + at, 4);
                    cp_async4(dst + S::kScales + (kTile + lane) * 4, p.cache.v_scale + at, 4);
                }
            } else {
                if (page_id == -2) record_error(p.ctrl, kErrInvalid);
                if (S::F8 && lane < kTile) {
                    float* scales = reinterpret_cast<float*>(ring + stage * S::kStage + S::kScales);
                    scales[lane] = 0.f, scales[kTile + lane] = 0.f;
                }
            }
            constexpr int kPerRow = S::kRow / 16;
            const int bytes = p.cache.dim * (S::F8 ? 1 : 2);
#pragma unroll
            for (int i = 0; i < kTile * kPerRow / 32; ++i) {
                const int c = i * 32 + lane, row = c / kPerRow, col = c % kPerRow * 16;
                const long long o = __shfl_sync(0xffffffffu, off, row);
                const bool in = o >= 0 && col < bytes;
                const long long src = in ? o + col : 0;
                cp_async16(dst + row * S::kPitch + col, p.cache.k + src, in ? 16 : 0);
                cp_async16(dst + (kTile + row) * S::kPitch + col, p.cache.v + src, in ? 16 : 0);
            }
            if (lane == 0) {
                const int last = put.first + put.count - 1;
                *reinterpret_cast<int4*>(ring + stage * S::kStage + S::kMeta) =
                    make_int4(put.b, put.vh, put.tile | (put.tile == put.first ? 1 << 30 : 0) | (put.tile == last ? 1 << 31 : 0), put.len);
            }
            put.next(p, heads);
            find_page();
        }
        cp_commit();
    };
    if (tiles > 0) {
        find_page();
        for (int s = 0; s < kStages - 1; ++s) fetch(s);

        float4 o[NT][JT];
        uint32_t q[NT][JT][2];
        float m[NT][2], l[NT][2], q_unit[NT][2];
        long long seg_first = 0;
        bool began = false, fresh = true;
        int stage = 0;
        for (long long it = 0; it < tiles; ++it) {
            cp_wait<kStages - 2>();
            __syncwarp();
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            const uint8_t* st = ring + stage * S::kStage;
            const uint32_t st_u = ring_u + stage * S::kStage;
            const int4 meta = *reinterpret_cast<const int4*>(st + S::kMeta);
            const int b = meta.x, vh = meta.y, tile = meta.z & 0x3fffffff, len = meta.w;
            const int head0 = vh / per_head * p.group + vh % per_head * S::kHeads;
            const int n_heads = min(S::kHeads, p.group - vh % per_head * S::kHeads);
            if (fresh) {
                // the segment's queries
                fresh = false;
                began = meta.z & (1 << 30);
                int f;
                tiles_of<kTile>(p, len, f);
                seg_first = s_start[warp].at + it - (tile - f);
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

            // scores: rows lane / 4 and + 8 of each 16, heads 2 (lane % 4) and + 1
            float4 s[NT][MT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) s[nt][mt] = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t k_at = st_u + (lane & 15) * S::kPitch + (lane >> 4) * 16;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (S::F8) {
#pragma unroll
                    for (int j = 0; j < JT; j += 2) {
                        uint32_t a[4];
                        ldsm(a, k_at + mt * 16 * S::kPitch + j * 16);
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
                        ldsm(a, k_at + mt * 16 * S::kPitch + j * 32);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma<false>(s[nt][mt], a[0], a[1], a[2], a[3], q[nt][j][0], q[nt][j][1]);
                    }
                }
            }
            // rows of this tile that count
            const int lo = (p.window && len > p.window ? len - p.window : 0) - tile * kTile, hi = len - tile * kTile;
            const float* scales = reinterpret_cast<const float*>(st + S::kScales);
            float vs[MT][2], vl[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = mt * 16 + i * 8 + (lane >> 2);
                    const bool in = r >= lo && r < hi;
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
                        x = in ? x * (q_unit[nt][0] * ks) : -INFINITY;
                        y = in ? y * (q_unit[nt][1] * ks) : -INFINITY;
                    }
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
            const uint32_t v_at = st_u + kTile * S::kPitch;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (S::F8) {
                    const uint32_t at = v_at + (mt * 16 + (lane & 15)) * S::kPitch + (lane >> 4) * 16;
#pragma unroll
                    for (int j = 0; j < JT; j += 2) {
                        uint32_t a[4];
                        ldsm_t(a, at + j * 16);
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
                    const uint32_t at = v_at + (mt * 16 + (lane & 7) + (lane >> 4) * 8) * S::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
                    for (int j = 0; j < JT; ++j) {
                        uint32_t a[4];
                        ldsm_t(a, at + j * 32);
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
#pragma unroll
                        for (int j = 0; j < JT; ++j) {
                            const float4 v = o[nt][j];
                            store_one<S>(p, b, head0 + nt * 8, n_heads - nt * 8, j, lane, make_float4(v.x * i0, v.y * i1, v.z * i0, v.w * i1));
                        }
                        const int h = nt * 8 + 2 * (lane & 3);
                        if (p.lse && lane < 4) {
                            float* lse = p.lse + static_cast<long long>(b) * p.Hq + head0;
                            if (h < n_heads) lse[h] = lse_of<S>(m[nt][0], l[nt][0]);
                            if (h + 1 < n_heads) lse[h + 1] = lse_of<S>(m[nt][1], l[nt][1]);
                        }
                    }
                } else {
                    // what began before this share first, what goes on behind it second
                    const int which = began ? 1 : 0;
                    float* part = scratch + which * S::kPart;
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
                        Open& w = s_open[warp * 2 + which];
                        w.first = seg_first;
                        w.end = seg_first + tiles_of<kTile>(p, len, f);
                        w.b = b, w.vh = vh;
                    }
                }
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
    }
    __syncthreads();

    // ---------------------------------------------------------------- joins
    const long long cta_from = static_cast<long long>(cta) * S::kWarps * total / warps, cta_to = (static_cast<long long>(cta) + 1) * S::kWarps * total / warps;
    const float* const cta_scratch = p.part + static_cast<long long>(cta) * S::kWarps * 2 * S::kPart;
    float* const cta_parts = p.part + static_cast<long long>(gridDim.x) * S::kWarps * 2 * S::kPart;
    for (int i = 0; i < 2 * S::kWarps;) {
        const Open seg = s_open[i];
        if (seg.end == 0) {
            ++i;
            continue;
        }
        // its parts: this CTA's open slots that follow with the same segment
        int n = 1, next = i + 1, slot[S::kWarps];
        slot[0] = i;
        for (; next < 2 * S::kWarps; ++next) {
            const Open& w = s_open[next];
            if (w.end == 0) continue;
            if (w.first != seg.first) break;
            slot[n++] = next;
        }
        i = next;
        const int head0 = seg.vh / per_head * p.group + seg.vh % per_head * S::kHeads;
        const int n_heads = min(S::kHeads, p.group - seg.vh % per_head * S::kHeads);
        const auto finish = [&](int e, int nt, int j, int ln, float4 o, float l0, float l1) {
            const float i0 = over<S>(l0), i1 = over<S>(l1);
            store_one<S>(p, seg.b, head0 + nt * 8, n_heads - nt * 8, j, ln, make_float4(o.x * i0, o.y * i1, o.z * i0, o.w * i1));
        };
        const auto finish_stats = [&](int h, float m0, float m1, float l0, float l1) {
            if (!p.lse) return;
            float* lse = p.lse + static_cast<long long>(seg.b) * p.Hq + head0;
            if (h < n_heads) lse[h] = lse_of<S>(m0, l0);
            if (h + 1 < n_heads) lse[h + 1] = lse_of<S>(m1, l1);
        };
        const auto own_part = [&](int k) { return cta_scratch + static_cast<long long>(slot[k]) * S::kPart; };
        if (seg.first >= cta_from && seg.end <= cta_to) {
            join<S>(n, own_part, finish, finish_stats);
            continue;
        }
        float* part = cta_parts + (2 * cta + (seg.first <= cta_from ? 0 : 1)) * static_cast<long long>(S::kPart);
        join<S>(
            n, own_part, [&](int e, int, int, int, float4 o, float, float) { reinterpret_cast<float4*>(part)[e] = o; },
            [&](int h, float m0, float m1, float l0, float l1) {
                *reinterpret_cast<float2*>(part + S::kFrag * 4 + h) = make_float2(m0, m1);
                *reinterpret_cast<float2*>(part + S::kFrag * 4 + S::kHeads + h) = make_float2(l0, l1);
            });
        // the CTA of a tile: the last one whose share begins at it or before
        const int c0 = static_cast<int>(((seg.first + 1) * ctas - 1) / total), c1 = static_cast<int>((seg.end * ctas - 1) / total);
        __syncthreads();
        if (tid == 0) {
            int* counter = p.counter + c0;
            const bool last = ptx::atom_add_acq_rel_gpu(counter, 1) == c1 - c0;
            if (last) ptx::st_relaxed_gpu(counter, 0);
            s_last = last;
        }
        __syncthreads();
        if (s_last) {
            const bool whole = seg.first == static_cast<long long>(c0) * S::kWarps * total / warps;
            const auto part_of = [&](int k) {
                return cta_parts + (2 * (c0 + k) + (k == 0 && !whole ? 1 : 0)) * static_cast<long long>(S::kPart);
            };
            join<S>(c1 - c0 + 1, part_of, finish, finish_stats);
        }
        __syncthreads();
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
long long parts_bytes(int num_sms)
{
    return 4LL * S::kPart * num_sms * 2 * (S::kWarps + 1);
}

}  // namespace

long long attn_decode_workspace(int group, int dim, int num_sms)
{
    const auto bytes = [&](auto s) { return parts_bytes<decltype(s)>(num_sms); };
    const long long a = with_shape(dim, false, group, bytes), b = with_shape(dim, true, group, bytes);
    return a > b ? a : b;
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
