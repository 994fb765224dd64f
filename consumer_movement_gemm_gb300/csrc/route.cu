// route.cu -- router logits -> the k experts of each token and their weights.
//
// Softmax and top-k in one pass over the logits.  L lanes (a power of two)
// share a token and hold V consecutive logits each as unsigned keys in the
// logits' order.  Every lane sorts its keys once (a merge network); each of
// the k steps then takes the largest head of the group and the lane that held
// it moves its list up.  Equal logits: the lowest expert first.  A bf16 logit
// and its expert's number fit one 32-bit key, so equal keys cannot occur; an
// fp32 logit's key carries its number beside it, and the lowest lane with the
// largest head wins.
//
// Masked experts (-inf or NaN) get the lowest keys and are recognised when
// they come up.  The results of a warp's tokens meet in shared memory, where
// exp and the sums are computed once per result, and leave as whole rows.
//
// What bounds it: integer instructions (half rate), 4 of them a logit for the
// keys and about 5 for the sort; the loads of four tokens a warp are in flight
// before the first is worked on.  65536 x 256 bf16, k = 8: 18.8 us, integer pipe
// 84 % busy (fp32 42 us); 40000 x 384 bf16, k = 16: 50 us; 1 x 32: 2.5 us, a launch.
#include <cuda_bf16.h>
#include "common.cuh"
#include "ops.cuh"

namespace tovl {

namespace {

constexpr int kWarps = 4;      // of a CTA

// Order-preserving key of an fp32 logit; 0 = masked.  -0 and +0 share a key.
__device__ __forceinline__ uint32_t to_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.f);
    if ((u & 0x7fffffffu) > 0x7f800000u || u == 0xff800000u) return 0;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float from_key(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// Two bf16 logits as order-preserving 16-bit keys: NaN becomes -inf, -0
// becomes +0, negative numbers are inverted, the others get the sign bit.
// -inf has key 0x007f.
__device__ __forceinline__ uint32_t to_keys(uint32_t pair)
{
    const uint32_t low = 0xff80ff80u, zero = 0u;
    __nv_bfloat162 v = reinterpret_cast<const __nv_bfloat162&>(pair);
    v = __hmax2(v, reinterpret_cast<const __nv_bfloat162&>(low));
    v = __hadd2(v, reinterpret_cast<const __nv_bfloat162&>(zero));
    const uint32_t u = reinterpret_cast<const uint32_t&>(v);
    return u ^ (((u >> 15) & 0x00010001u) * 0xffffu | 0x80008000u);
}

// exp(v - m), m the largest logit: 1 where they are equal (also at +inf), 0
// where the expert is masked
__device__ __forceinline__ float weight_of(float v, float m)
{
    return v == -INFINITY ? 0.f : v == m ? 1.f : expf(v - m);
}

template <bool F32>
struct Key {
    uint32_t k;
    uint32_t idx;       // F32 only
    // does this key come before o?
    __device__ __forceinline__ bool before(const Key& o) const { return F32 ? k > o.k || (k == o.k && idx < o.idx) : k > o.k; }
};

template <bool F32>
__device__ __forceinline__ void order(Key<F32>& a, Key<F32>& b)
{
    if constexpr (F32) {
        const bool swap = b.before(a);
        const Key<F32> x = a;
        a.k = swap ? b.k : a.k, a.idx = swap ? b.idx : a.idx;
        b.k = swap ? x.k : b.k, b.idx = swap ? x.idx : b.idx;
    } else {
        const uint32_t x = a.k;
        a.k = max(x, b.k);
        b.k = min(x, b.k);
    }
}

// Odd-even merge sort, first come first.
template <bool F32, int V>
__device__ __forceinline__ void sort_keys(Key<F32> (&key)[V])
{
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(key[i + j], key[i + j + k]);
}

template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    if constexpr (L == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int d = L / 2; d; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
}

// Tokens of a warp: 32 / L at a time, and at least four in all.
template <int L>
constexpr int kSets = L <= 8 ? 1 : L / 8;

template <int L, int V, bool F32, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteParams p)
{
    extern __shared__ float stage[];      // per warp [tokens][k]: keys, experts, weights; then sums [tokens]
    constexpr int kTok = 32 / L, kAll = kTok * kSets<L>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & (L - 1), tok = lane / L;
    const long long t0 = (static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp) * kAll;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (t0 >= p.T) return;
    uint32_t* sk = reinterpret_cast<uint32_t*>(stage) + warp * (kAll * (3 * p.k + 1));
    int* si = reinterpret_cast<int*>(sk + kAll * p.k);
    float* sw = reinterpret_cast<float*>(sk + 2 * kAll * p.k);
    float* sums = sw + kAll * p.k;
    const int left = p.E - sub * V;       // elements of this lane
    constexpr int kPer = F32 ? 4 : 8, kWords = V / kPer;
    uint4 raw[kSets<L>][kWords];
    const char* base[kSets<L>];
#pragma unroll
    for (int s = 0; s < kSets<L>; ++s) {
        const long long t = t0 + s * kTok + tok;
        base[s] = static_cast<const char*>(p.logits) + ((t < p.T ? t : t0) * p.ld + sub * V) * (F32 ? 4 : 2);
        if (VEC) {
#pragma unroll
            for (int c = 0; c < kWords; ++c) {
                const uint32_t none = F32 ? 0xff800000u : 0xff80ff80u;
                raw[s][c] = make_uint4(none, none, none, none);
                if (c * kPer < left) raw[s][c] = __ldg(reinterpret_cast<const uint4*>(base[s]) + c);
            }
        }
    }
#pragma unroll
    for (int s = 0; s < kSets<L>; ++s) {
        Key<F32> key[V];
        if constexpr (F32) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t w[4] = {raw[s][v / 4].x, raw[s][v / 4].y, raw[s][v / 4].z, raw[s][v / 4].w};
                float f = __uint_as_float(w[v & 3]);
                if (!VEC) f = v < left ? __ldg(reinterpret_cast<const float*>(base[s]) + v) : -INFINITY;
                key[v].k = to_key(f);
                key[v].idx = sub * V + v;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                const uint32_t w[4] = {raw[s][v / 8].x, raw[s][v / 8].y, raw[s][v / 8].z, raw[s][v / 8].w};
                uint32_t pair = w[(v / 2) & 3];
                if (!VEC) {
                    const uint16_t* at = reinterpret_cast<const uint16_t*>(base[s]);
                    pair = (v < left ? __ldg(at + v) : 0xff80u) | (v + 1 < left ? __ldg(at + v + 1) : 0xff80u) << 16;
                }
                const uint32_t two = to_keys(pair), number = 0xffffu - (sub * V + v);
                key[v].k = two << 16 | number;
                key[v + 1].k = (two & 0xffff0000u) | (number - 1);
            }
        }
        if (!p.renormalize) {
            // the sum over all experts, relative to the largest logit
            uint32_t top = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) top = max(top, key[v].k);
            top = group_max<L>(top);
            const auto value = [](uint32_t k) {
                if (F32) return k ? from_key(k) : -INFINITY;
                return from_key(k & 0xffff0000u | ((k & 0x80000000u) ? 0u : 0xffffu));
            };
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += weight_of(value(key[v].k), value(top));
#pragma unroll
            for (int d = L / 2; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (sub == 0) sums[s * kTok + tok] = sum;
        }
        sort_keys<F32, V>(key);
        const int at = (s * kTok + tok) * p.k;
        // one step: the largest head leaves, its lane's list moves up by one;
        // `keep` of its elements can still be needed
        const auto step = [&](int j, int keep) {
            const uint32_t best = group_max<L>(key[0].k);
            bool mine = key[0].k == best;
            if (F32) {
                uint32_t who = __ballot_sync(0xffffffffu, mine);
                if (L < 32) who = (who >> (tok * L)) & ((1u << (L & 31)) - 1u);
                mine = sub == __ffs(who) - 1;
                if (mine) si[at + j] = best == 0 ? -1 : static_cast<int>(key[0].idx);
            }
            if (sub == (j & (L - 1))) sk[at + j] = best;
#pragma unroll
            for (int v = 0; v + 1 < V; ++v)
                if (v < keep) {
                    key[v].k = mine ? key[v + 1].k : key[v].k;
                    if (F32) key[v].idx = mine ? key[v + 1].idx : key[v].idx;
                }
            if (keep >= V) key[V - 1].k = mine ? 0 : key[V - 1].k;
        };
        if (p.k <= V) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < p.k) step(j, V - 1 - j);
        } else {
#pragma unroll 1
            for (int j = 0; j < p.k; ++j) step(j, V);
        }
    }
    __syncwarp();
    // a result's logit from its key, and its weight relative to the token's largest
    const int n_tok = static_cast<int>(min(static_cast<long long>(kAll), p.T - t0)), n = n_tok * p.k;
    const auto value = [](uint32_t k) {
        if (F32) return k ? from_key(k) : -INFINITY;
        return k < 0x00800000u ? -INFINITY : from_key((k & 0xffff0000u) | ((k & 0x80000000u) ? 0u : 0xffffu));
    };
    for (int i = lane; i < n; i += 32) {
        const uint32_t k = sk[i];
        if (!F32) si[i] = k < 0x00800000u ? -1 : static_cast<int>(0xffffu - (k & 0xffffu));
        sw[i] = weight_of(value(k), value(sk[i / p.k * p.k]));
    }
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
        const int token = i / p.k;
        float sum = 0.f;
        if (p.renormalize)
            for (int j = 0; j < p.k; ++j) sum += sw[token * p.k + j];
        else sum = sums[token];
        p.gate_w[t0 * p.k + i] = sw[i] > 0.f ? sw[i] / sum : 0.f;
        p.topk[t0 * p.k + i] = si[i];
    }
}

template <int L, int V>
cudaError_t launch(const RouteParams& p, cudaStream_t stream, bool pdl)
{
    constexpr int kAll = 32 / L * kSets<L>;
    const int es = p.f32 ? 4 : 2;
    const bool vec = p.E % (16 / es) == 0 && p.ld % (16 / es) == 0 && (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0;
    cudaLaunchConfig_t lc = {};
    // (32 tokens a warp with more than 16 slots each would take over 48 KB)
    const int warps = p.k > 16 ? kWarps / 2 : kWarps;
    lc.gridDim = dim3((p.T - 1) / (warps * kAll) + 1);
    lc.blockDim = dim3(warps * 32);
    lc.dynamicSmemBytes = warps * kAll * (3 * p.k + 1) * 4;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = pdl ? 1 : 0;
    if (p.f32) return vec ? cudaLaunchKernelEx(&lc, route_kernel<L, V, true, true>, p)
                          : cudaLaunchKernelEx(&lc, route_kernel<L, V, true, false>, p);
    return vec ? cudaLaunchKernelEx(&lc, route_kernel<L, V, false, true>, p)
               : cudaLaunchKernelEx(&lc, route_kernel<L, V, false, false>, p);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream, bool pdl)
{
    if (p.E <= 8) return launch<1, 8>(p, stream, pdl);
    if (p.E <= 16) return launch<2, 8>(p, stream, pdl);
    if (p.E <= 32) return launch<4, 8>(p, stream, pdl);
    if (p.E <= 64) return launch<8, 8>(p, stream, pdl);
    if (p.E <= 128) return launch<16, 8>(p, stream, pdl);
    if (p.E <= 256) return launch<32, 8>(p, stream, pdl);
    return launch<32, 16>(p, stream, pdl);
}

}  // namespace tovl
