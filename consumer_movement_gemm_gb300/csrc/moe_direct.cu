// moe_direct.cu -- the expert layer of moe_decode.cu where its time is latency:
// two kernels without rings, counters or grid barriers (use_direct_moe is the
// rule).
//
// The first gives h = silu(x W13[e][:, :I]) * (x W13[e][:, I:]), a CTA 32 (4-bit
// weights: 16) of its columns for one expert, gate and up columns side by side
// in one tile.  The second gives 64 (32) columns of the result, the sums over
// all experts and rows of W2 shared out to its warps as one list; a warp adds
// what it has to the CTA's sums in shared memory, times the gate weight, each
// time its expert changes.  Warps read their weights straight into registers,
// a block ahead of the one that is multiplied; with few tiles a cluster of two
// or four CTAs shares out the rows and its first CTA gets the others' sums.  The
// second kernel reads the routing and its first weights while the first ends.
//
// Eight tokens at a time (of more than eight, sixteen) are the columns of the
// tensor core's second operand, whether or not they name the expert (zeros, and
// their results dropped), so nothing is gathered.  More tokens are more CTAs,
// which find the weights of experts that they share in L2.
//
// h is fp32 in memory.  With bf16 weights it enters the second product as two
// bf16 numbers, its rounding and the rest; with 4-bit weights as fp16 with a
// power of two per 128 columns.  Sums are fp32, in a fixed order.
//
// What bounds it: at small sizes two launches and a CTA's dependent loads (1
// token, 256 x 128: 5.2 us, 1024 x 512: 7.4, through the rings 14.4 and 19.2); at
// large ones the bytes in flight, one block a warp, and the start of two grids (1
// token, 2 of 8 experts of 4096 x 2048, bf16: 23.9 us, 4.2 TB/s, of 4096 x 4096: 39.9,
// 5.0 TB/s; through the rings 30.6 and 43.9).  Two blocks a warp spill registers:
// 27.1 us for the first.
#include <type_traits>
#include "launch.cuh"
#include "skinny.cuh"

namespace tovl {

namespace {

using namespace skinny;

constexpr int kWarps = 16;             // at most; CTAs of 8 share an SM
constexpr int kMaxTokens = 16;
constexpr int kCluster = 4;
constexpr int kMaxActive = kMaxTokens * kMaxDecodeK;

struct Routing {
    uint32_t mask[kMaxExperts];        // tokens of each expert
    int id[kMaxTokens * kMaxDecodeK];
    float gate[kMaxTokens * kMaxDecodeK];
    int active[kMaxActive];            // the experts with tokens, ascending
    int n;
};

// Routing of the tokens t0 .. t0 + cnt.  False if an id (of any token) is
// outside [-1, E).
__device__ bool read_routing(const MoeDirectParams& p, Routing& rt, int t0, int cnt)
{
    const int tid = threadIdx.x;
    bool bad = false;
    for (int i = tid; i < p.T * p.k; i += blockDim.x) {
        const int e = __ldcg(p.topk + i);
        bad |= e < -1 || e >= p.E;
    }
    for (int e = tid; e < p.E; e += blockDim.x) rt.mask[e] = 0;
    const bool own = tid < cnt * p.k;      // (256 threads at least)
    int id = -1;
    if (own) {
        id = __ldcg(p.topk + t0 * p.k + tid);
        rt.id[tid] = id;
        rt.gate[tid] = __ldcg(p.gate_w + t0 * p.k + tid);
    }
    if (__syncthreads_or(bad)) return false;
    if (id >= 0) atomicOr(rt.mask + id, 1u << (tid / p.k));
    __syncthreads();
    if (tid < 32) {
        int n = 0;
        for (int base = 0; base < p.E; base += 32) {
            const bool on = base + tid < p.E && rt.mask[base + tid];
            const uint32_t m = __ballot_sync(0xffffffffu, on);
            if (on) rt.active[n + __popc(m & ((1u << tid) - 1))] = base + tid;
            n += __popc(m);
        }
        if (tid == 0) rt.n = n;
    }
    __syncthreads();
    return true;
}

// The slot of token t that names e first (-1: none), and the weights of all that do.
__device__ __forceinline__ int find_slot(const MoeDirectParams& p, const Routing& rt, int t, int e, float& gate)
{
    int first = -1;
    gate = 0.f;
    for (int j = 0; j < p.k; ++j)
        if (rt.id[t * p.k + j] == e) {
            if (first < 0) first = j;
            gate += rt.gate[t * p.k + j];
        }
    return first;
}

// A lane's part of a block of weights.  bf16: rows 8t .. 8t + 7 of 32, eight
// columns.  4-bit: octet rows t, t + 4, .. of 128 rows, four columns.
template <int G, bool Z>
struct Weights {
    static constexpr int kRows = 128, kLaneCols = 4, kGroups = 128 / G;
    uint4 w[4];
    uint2 scale[kGroups];
    uint32_t zero[kGroups];

    __device__ __forceinline__ void load(const MoeWeights& m, int e, int b, int K, int N, int n, bool col, int t)
    {
        const long long row = static_cast<long long>(e) * (K / 8);
#pragma unroll
        for (int R = 0; R < 4; ++R) {
            const int octet = b * 16 + 4 * R + t;
            w[R] = make_uint4(0, 0, 0, 0);
            if (col && octet * 8 < K) w[R] = ld_stream(static_cast<const uint32_t*>(m.w) + (row + octet) * N + n);
        }
        const long long group = static_cast<long long>(e) * (K / G) + b * kGroups;
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            const bool in = col && b * 128 + q * G < K;
            const long long at = (group + q) * N + n;
            scale[q] = in ? __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(m.scale) + at)) : make_uint2(0, 0);
            zero[q] = Z && in ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(m.zero) + at)) : 0u;
        }
    }
};
template <>
struct Weights<0, false> {
    static constexpr int kRows = 32, kLaneCols = 8;
    uint4 w[8];

    __device__ __forceinline__ void load(const MoeWeights& m, int e, int b, int K, int N, int n, bool col, int t)
    {
        const int k = b * 32 + 8 * t;
        const __nv_bfloat16* at = static_cast<const __nv_bfloat16*>(m.w) + (static_cast<long long>(e) * K + k) * N + n;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            w[r] = col && k < K ? ld_stream(reinterpret_cast<const uint32_t*>(at + static_cast<long long>(r) * N)) : make_uint4(0, 0, 0, 0);
    }
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Sums of a warp: token columns 2t, 2t + 1 of each eight, of the lane group's
// four or eight weight columns.
template <int NT, int G, bool Z>
struct Sums {
    static constexpr int kTiles = G ? 2 : 4;
    static constexpr int kCols = G ? 32 : 64;
    float v[kTiles][NT][4];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[m][nt][i] = 0.f;
    }

    // bf16: two steps of 16 rows, column pair m of the lanes is the tile m; the rows'
    // pairs of a column come out of two rows' words by byte permutation
    template <bool LO>
    __device__ __forceinline__ void add(const Weights<0, false>& a, const uint4 (&b)[NT], const uint4 (&lo)[NT])
    {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t r0 = word(a.w[4 * s], m), r1 = word(a.w[4 * s + 1], m);
                const uint32_t r2 = word(a.w[4 * s + 2], m), r3 = word(a.w[4 * s + 3], m);
                const uint32_t a0 = __byte_perm(r0, r1, 0x5410), a1 = __byte_perm(r0, r1, 0x7632);
                const uint32_t a2 = __byte_perm(r2, r3, 0x5410), a3 = __byte_perm(r2, r3, 0x7632);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma(v[m][nt], a0, a1, a2, a3, s ? b[nt].z : b[nt].x, s ? b[nt].w : b[nt].y);
                    if (LO) mma(v[m][nt], a0, a1, a2, a3, s ? lo[nt].z : lo[nt].x, s ? lo[nt].w : lo[nt].y);
                }
            }
    }

    // column 0 .. of the lane group for token 8 nt + 2t + j, four of them (half: the next four)
    __device__ __forceinline__ float4 four(int nt, int j, int half) const
    {
        const int m = half * 2;
        return make_float4(v[m][nt][j], v[m][nt][j + 2], v[m + 1][nt][j], v[m + 1][nt][j + 2]);
    }
};

// The warps' sums of a CTA, [token][column] a warp.  Fours of columns are
// stored by (half, group ^ 2t), which keeps a quarter warp's in different banks.
template <int NT, int COLS>
struct Joined {
    float red[kWarps][NT * 8][COLS];
    float join[kCluster - 1][NT * 8][COLS];

    static __device__ __forceinline__ int four_of(int g, int half, int t) { return half * 8 + (g ^ (2 * t)); }
    static __device__ __forceinline__ int place(int r, int c)
    {
        const int g = COLS == 64 ? c >> 3 : c >> 2, half = COLS == 64 ? (c >> 2) & 1 : 0;
        return four_of(g, half, (r >> 1) & 3) * 4 + (c & 3);
    }
    __device__ __forceinline__ float4& at(int warp, int g, int t, int nt, int j, int half)
    {
        return *reinterpret_cast<float4*>(&red[warp][nt * 8 + 2 * t + j][four_of(g, half, t) * 4]);
    }
    __device__ __forceinline__ float sum(int r, int c, int warps) const
    {
        const int at = place(r, c);
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps / 2; ++i) v += red[i][r][at];
        if (warps > kWarps / 2) {
#pragma unroll
            for (int i = kWarps / 2; i < kWarps; ++i) v += red[i][r][at];
        }
        return v;
    }
    // The CTA's sums to the first CTA of the cluster.  False in the others.
    __device__ __forceinline__ bool gather(int rank, int split, int rows, int warps)
    {
        if (split == 1) return true;
        __syncwarp();
        ptx::cluster_wait();           // the first CTA runs
        if (rank > 0)
            for (int i = threadIdx.x; i < rows * COLS; i += blockDim.x) {
                const int r = i / COLS, c = i % COLS;
                st_cluster_f32(ptx::mapa_shared(ptx::smem_u32(&join[rank - 1][r][c]), 0), sum(r, c, warps));
            }
        __syncwarp();
        ptx::cluster_sync();
        return rank == 0;
    }
    __device__ __forceinline__ float total(int r, int c, int split, int warps) const
    {
        float v = sum(r, c, warps);
        for (int i = 1; i < split; ++i) v += join[i - 1][r][c];
        return v;
    }
};

__device__ __forceinline__ uint32_t max_exponent(const float4& v)
{
    const uint32_t a = max(__float_as_uint(v.x) & 0x7f800000u, __float_as_uint(v.y) & 0x7f800000u);
    const uint32_t b = max(__float_as_uint(v.z) & 0x7f800000u, __float_as_uint(v.w) & 0x7f800000u);
    return max(a, b) >> 23;
}

// Scale of this lane's token g to those of the sums' tokens 2t and 2t + 1.
__device__ __forceinline__ float2 of_sums(float v, int t)
{
    return make_float2(__shfl_sync(0xffffffffu, v, 8 * t), __shfl_sync(0xffffffffu, v, 8 * t + 4));
}

// Largest of a lane's four (its token's part of 128 columns).
__device__ __forceinline__ uint32_t max_of_token(uint32_t e)
{
    e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
    return max(e, __shfl_xor_sync(0xffffffffu, e, 2));
}

// Two numbers as bf16 pairs: their roundings and what those left over (nothing,
// where a number has overflowed).
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo)
{
    hi = ptx::pack_bf16x2(a, b);
    const float da = a - bf16_lo(hi), db = b - bf16_hi(hi);
    lo = ptx::pack_bf16x2(fabsf(da) < INFINITY ? da : 0.f, fabsf(db) < INFINITY ? db : 0.f);
}

// grid: tiles of columns, CTAs of a cluster, (NT * 8 tokens, expert of theirs)
template <int NT, int G, bool Z>
__global__ void __launch_bounds__(kWarps * 32, 1) moe_up_kernel(const __grid_constant__ MoeDirectParams p, int most_active)
{
    using W = Weights<G, Z>;
    using S = Sums<NT, G, Z>;
    using J = Joined<NT, S::kCols>;
    constexpr int kHalf = S::kCols / 2, kOctets = W::kRows / 32;
    __shared__ Routing rt;
    extern __shared__ __align__(16) uint8_t smem[];
    J& sums = *reinterpret_cast<J*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5, split = gridDim.y, rank = blockIdx.y;
    const int t0 = blockIdx.z / most_active * (NT * 8), cnt = min(NT * 8, p.T - t0), a = blockIdx.z % most_active;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    int e;
    uint32_t named;                    // tokens that name e
    if (p.T <= NT * 8 && p.T * p.k <= 32) {
        // One name a lane: every warp finds the expert by itself, without a barrier
        // before the first weights (1 token, 1024 x 512: 7.8 -> 7.4 us); the experts
        // in the order of their first names.  Of a call whose tokens are all here
        // (t0 = 0): tokens and names are counted from the call's first.
        const int id = lane < p.T * p.k ? __ldcg(p.topk + lane) : -1;
        const float weight = lane < p.T * p.k ? __ldcg(p.gate_w + lane) : 0.f;
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        const uint32_t firsts = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
        if (__any_sync(0xffffffffu, id < -1 || id >= p.E)) {
            if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) record_error(p.ctrl, kErrInvalid);
            return;
        }
        if (a >= __popc(firsts)) return;
        const int first = __fns(firsts, 0, a + 1);
        e = __shfl_sync(0xffffffffu, id, first);
        const bool mine = lane < p.T * p.k && id == e;
        named = __reduce_or_sync(0xffffffffu, mine ? 1u << (lane / p.k) : 0u);
        if (warp == 0 && lane < p.T * p.k) {       // (read after the next barrier)
            rt.id[lane] = id;
            rt.gate[lane] = weight;
        }
    } else {
        if (!read_routing(p, rt, t0, cnt)) {
            if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) record_error(p.ctrl, kErrInvalid);
            return;
        }
        if (a >= rt.n) return;
        e = rt.active[a];
        named = rt.mask[e];
    }
    __syncwarp();
    if (split > 1) ptx::cluster_arrive_relaxed();
    const uint32_t use = named >> g;
    const int i0 = blockIdx.x * kHalf, in_half = i0 + (g & 3) * W::kLaneCols, n = (g >> 2) * p.I + in_half;
    const bool col = in_half < p.I;
    const int blocks = (p.H + W::kRows - 1) / W::kRows, stride = warps * split;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + (t0 + g) * p.ldx;
    const auto octet = [&](int b, int R, int nt) {
        const int k = b * W::kRows + 32 * R + 8 * t;
        return (use >> (8 * nt) & 1) && k < p.H ? __ldg(reinterpret_cast<const uint4*>(x + nt * 8 * p.ldx + k)) : make_uint4(0, 0, 0, 0);
    };
    constexpr bool kRowsAhead = NT == 1;       // (more would not fit the registers)
    S acc;
    acc.clear();
    W next;
    uint4 next_x[kOctets];
    const auto fetch = [&](int b) {
        next.load(p.up, e, b, p.H, 2 * p.I, n, col, t);
        if (kRowsAhead) {
#pragma unroll
            for (int R = 0; R < kOctets; ++R) next_x[R] = octet(b, R, 0);
        }
    };
    int b = rank * warps + warp;
    if (b < blocks) fetch(b);
    for (; b < blocks; b += stride) {
        const W w = next;
        uint4 xb[kOctets][NT];
#pragma unroll
        for (int R = 0; R < kOctets; ++R)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) xb[R][nt] = kRowsAhead ? next_x[R] : octet(b, R, nt);
        if (b + stride < blocks) fetch(b + stride);
        if constexpr (G == 0) {
            acc.template add<false>(w, xb[0], xb[0]);
        } else {
            float2 sx[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t ex = 0;
#pragma unroll
                for (int R = 0; R < 4; ++R) ex = max(ex, skinny::max_exponent(xb[R][nt]));
                ex = max_of_token(ex);
                const float f = half_scale(ex);
#pragma unroll
                for (int R = 0; R < 4; ++R) xb[R][nt] = bf16x8_to_half(xb[R][nt], f);
                sx[nt] = of_sums(half_unscale(ex), t);
            }
            multiply_q4<NT, G, Z>(
                acc.v, sx, [&](int R) { return w.w[R]; }, [&](int q) { return w.zero[q]; }, [&](int q) { return w.scale[q]; },
                [&](int R, int nt) { return xb[R][nt]; });
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int half = 0; half < S::kTiles / 2; ++half) sums.at(warp, g, t, nt, j, half) = acc.four(nt, j, half);
    __syncthreads();
    if (!sums.gather(rank, split, cnt, warps)) return;
    for (int i = threadIdx.x; i < cnt * kHalf; i += blockDim.x) {
        const int r = i / kHalf, c = i % kHalf;
        float gate;
        const int j = find_slot(p, rt, r, e, gate);
        if (j < 0 || i0 + c >= p.I) continue;
        const float v = sums.total(r, c, split, warps), u = sums.total(r, kHalf + c, split, warps);
        static_cast<float*>(p.h_hi)[((t0 + r) * p.k + j) * static_cast<long long>(p.I) + i0 + c] = v / (1.f + expf(-v)) * u;
    }
}

// grid: tiles of columns, CTAs of a cluster, NT * 8 tokens
template <int NT, int G, bool Z>
__global__ void __launch_bounds__(kWarps * 32, 1) moe_down_kernel(const __grid_constant__ MoeDirectParams p)
{
    using W = Weights<G, Z>;
    using S = Sums<NT, G, Z>;
    using J = Joined<NT, S::kCols>;
    constexpr int kOctets = W::kRows / 32;
    __shared__ Routing rt;
    extern __shared__ __align__(16) uint8_t smem[];
    J& sums = *reinterpret_cast<J*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5, split = gridDim.y, rank = blockIdx.y;
    const int t0 = blockIdx.z * (NT * 8), cnt = min(NT * 8, p.T - t0);
    // (what came before the first kernel is complete: that kernel has waited for
    // it before it let this one start)
    if (!read_routing(p, rt, t0, cnt)) {
        ptx::grid_dep_wait();
        return;
    }
    if (split > 1) ptx::cluster_arrive_relaxed();
    const int n = blockIdx.x * S::kCols + g * W::kLaneCols;
    const bool col = n < p.H;
    const int per = (p.I + W::kRows - 1) / W::kRows;      // blocks of an expert
    const int items = rt.n * per, share = rank * warps + warp, shares = warps * split;
    int item = items * share / shares;
    const int end = items * (share + 1) / shares;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int half = 0; half < S::kTiles / 2; ++half) sums.at(warp, g, t, nt, j, half) = make_float4(0.f, 0.f, 0.f, 0.f);
    W next;
    int a = item / per, b = item - a * per;
    if (item < end) next.load(p.down, rt.active[a], b, p.I, p.H, n, col, t);
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    S acc;
    acc.clear();
    int row[NT];                       // of h, of this lane's tokens for the expert; -1: they do not name it
    float gate[NT];
    bool fresh = true;
    for (; item < end; ++item) {
        const W w = next;
        if (fresh) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = nt * 8 + g, j = r < cnt ? find_slot(p, rt, r, rt.active[a], gate[nt]) : -1;
                row[nt] = j < 0 ? -1 : (t0 + r) * p.k + j;
                if (j < 0) gate[nt] = 0.f;
            }
        }
        int na = a, nb = b + 1;
        if (nb == per) na = a + 1, nb = 0;
        const bool more = item + 1 < end;
        // eight numbers of h of a token
        const auto octet = [&](int R, int nt, float4 (&v)[2]) {
            const int k = b * W::kRows + 32 * R + 8 * t;
            const float4* h = reinterpret_cast<const float4*>(static_cast<const float*>(p.h_hi) + row[nt] * static_cast<long long>(p.I) + k);
            const bool in = row[nt] >= 0 && k < p.I;
            v[0] = in ? __ldcg(h) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[1] = in ? __ldcg(h + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        if constexpr (G == 0) {
            float4 v[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) octet(0, nt, v[nt]);
            if (more) next.load(p.down, rt.active[na], nb, p.I, p.H, n, col, t);
            uint4 x[NT], rest[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                split_pair(v[nt][0].x, v[nt][0].y, x[nt].x, rest[nt].x);
                split_pair(v[nt][0].z, v[nt][0].w, x[nt].y, rest[nt].y);
                split_pair(v[nt][1].x, v[nt][1].y, x[nt].z, rest[nt].z);
                split_pair(v[nt][1].z, v[nt][1].w, x[nt].w, rest[nt].w);
            }
            acc.template add<true>(w, x, rest);
        } else {
            uint4 x[4][NT];
            float2 sx[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float4 v[4][2];
#pragma unroll
                for (int R = 0; R < 4; ++R) octet(R, nt, v[R]);
                if (nt == 0 && more) next.load(p.down, rt.active[na], nb, p.I, p.H, n, col, t);
                uint32_t ex = 0;
#pragma unroll
                for (int R = 0; R < 4; ++R) ex = max(ex, max(max_exponent(v[R][0]), max_exponent(v[R][1])));
                ex = max_of_token(ex);
                const float f = half_scale(ex);
#pragma unroll
                for (int R = 0; R < 4; ++R)
                    x[R][nt] = make_uint4(pack_h2(v[R][0].x * f, v[R][0].y * f), pack_h2(v[R][0].z * f, v[R][0].w * f),
                                          pack_h2(v[R][1].x * f, v[R][1].y * f), pack_h2(v[R][1].z * f, v[R][1].w * f));
                sx[nt] = of_sums(half_unscale(ex), t);
            }
            multiply_q4<NT, G, Z>(
                acc.v, sx, [&](int R) { return w.w[R]; }, [&](int q) { return w.zero[q]; }, [&](int q) { return w.scale[q]; },
                [&](int R, int nt) { return x[R][nt]; });
        }
        fresh = na != a;
        if (fresh || !more) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 gates = of_sums(gate[nt], t);
                const uint32_t named = __ballot_sync(0xffffffffu, row[nt] >= 0);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (named >> (8 * t + 4 * j) & 1) {
                        const float w1 = j ? gates.y : gates.x;
#pragma unroll
                        for (int half = 0; half < S::kTiles / 2; ++half) {
                            float4& s = sums.at(warp, g, t, nt, j, half);
                            const float4 v = acc.four(nt, j, half);
                            s = make_float4(fmaf(w1, v.x, s.x), fmaf(w1, v.y, s.y), fmaf(w1, v.z, s.z), fmaf(w1, v.w, s.w));
                        }
                    }
            }
            acc.clear();
        }
        a = na;
        b = nb;
    }
    __syncthreads();
    if (!sums.gather(rank, split, cnt, warps)) return;
    for (int i = threadIdx.x; i < cnt * S::kCols; i += blockDim.x) {
        const int r = i / S::kCols, c = i % S::kCols, at = blockIdx.x * S::kCols + c;
        if (at < p.H) static_cast<__nv_bfloat16*>(p.out)[(t0 + r) * p.ldo + at] = __float2bfloat16(sums.total(r, c, split, warps));
    }
}

// One CTA of 16 warps per SM where that is all of them, else CTAs of 8, two on
// an SM; clusters as long as they fit the SMs and leave each warp a block.
cudaLaunchConfig_t shape(cudaLaunchAttribute (&attr)[2], int tiles, int z, int blocks, int smem, int sms, cudaStream_t stream, bool pdl)
{
    const int warps = tiles * z <= sms ? kWarps : kWarps / 2;
    int split = 1;
    while (split < kCluster && tiles * z * split * 2 <= sms && split * warps < blocks) split *= 2;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(tiles, split, z);
    lc.blockDim = dim3(warps * 32);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    lc.attrs = attr;
    if (split > 1) {
        attr[lc.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[lc.numAttrs].val.clusterDim.x = 1;
        attr[lc.numAttrs].val.clusterDim.y = split;
        attr[lc.numAttrs].val.clusterDim.z = 1;
        ++lc.numAttrs;
    }
    if (pdl) {
        attr[lc.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[lc.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++lc.numAttrs;
    }
    return lc;
}

template <int NT, int G, bool Z>
cudaError_t launch(const MoeDirectParams& p, int sms, cudaStream_t stream, bool pdl)
{
    constexpr int kCols = Sums<NT, G, Z>::kCols, kRows = Weights<G, Z>::kRows;
    constexpr int kSmem = static_cast<int>(sizeof(Joined<NT, kCols>));
    const int passes = (p.T + NT * 8 - 1) / (NT * 8), names = (p.T < NT * 8 ? p.T : NT * 8) * p.k;
    const int active = names < p.E ? names : p.E;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t lc = shape(attr, (2 * p.I + kCols - 1) / kCols, passes * active, (p.H + kRows - 1) / kRows, kSmem, sms, stream, pdl);
    const cudaError_t e = cudaLaunchKernelEx(&lc, moe_up_kernel<NT, G, Z>, p, active);
    if (e != cudaSuccess) return e;
    lc = shape(attr, (p.H + kCols - 1) / kCols, passes, active * ((p.I + kRows - 1) / kRows), kSmem, sms, stream, pdl);
    return cudaLaunchKernelEx(&lc, moe_down_kernel<NT, G, Z>, p);
}

template <int NT, int G, bool Z>
cudaError_t prepare()
{
    constexpr int kSmem = static_cast<int>(sizeof(Joined<NT, Sums<NT, G, Z>::kCols>));
    const cudaError_t e = cudaFuncSetAttribute(moe_up_kernel<NT, G, Z>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(moe_down_kernel<NT, G, Z>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

// Calls f with the kernels' types: 8 or 16 tokens at a time, a group, zeros.
template <class F>
cudaError_t with_types(bool wide, int group, bool zero, F f)
{
    const auto zeros = [&](auto nt, auto g) {
        return zero ? f(nt, g, std::true_type()) : f(nt, g, std::false_type());
    };
    const auto groups = [&](auto nt) {
        if (group == 32) return zeros(nt, std::integral_constant<int, 32>());
        if (group == 64) return zeros(nt, std::integral_constant<int, 64>());
        if (group == 128) return zeros(nt, std::integral_constant<int, 128>());
        return f(nt, std::integral_constant<int, 0>(), std::false_type());
    };
    return wide ? groups(std::integral_constant<int, 2>()) : groups(std::integral_constant<int, 1>());
}

}  // namespace

cudaError_t prepare_moe_direct()
{
    for (int i = 0; i < 16; ++i) {
        const cudaError_t e = with_types(i & 1, (i >> 2) * 32 + (i >> 2 == 3 ? 32 : 0), i >> 1 & 1, [](auto nt, auto g, auto z) {
            return prepare<decltype(nt)::value, decltype(g)::value, decltype(z)::value>();
        });
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_moe_direct(const MoeDirectParams& p, int group, bool zero, int sms, cudaStream_t stream, bool pdl)
{
    return with_types(p.T > 8, group, zero, [&](auto nt, auto g, auto z) {
        return launch<decltype(nt)::value, decltype(g)::value, decltype(z)::value>(p, sms, stream, pdl);
    });
}

}  // namespace tovl
