// route.cu -- router logits -> the k experts of each token and their weights.
//
// Softmax and top-k in one pass over the logits.  L lanes (a power of two)
// share a token and hold up to V = 8 or 16 consecutive logits each, as
// unsigned keys whose order is the logits' order; key 0 is a masked expert (-inf or
// NaN), which is never chosen.  Each of the k steps takes the largest key of
// the group, the lowest lane that holds it and that lane's first element with
// it -- the lowest expert index among equals -- and strikes it out.  The
// results of a warp's tokens meet in shared memory and leave as whole rows.
#include <cuda_bf16.h>
#include "common.cuh"
#include "ops.cuh"

namespace tovl {

namespace {

constexpr int kWarps = 4;

// Order-preserving key of a logit; 0 = masked.  -0 and +0 share a key.
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

// exp(v - m) of a logit's key, m the largest logit: 1 where they are equal
// (also at +inf), 0 where the expert is masked
__device__ __forceinline__ float weight_of(uint32_t key, uint32_t top)
{
    if (key == 0) return 0.f;
    return key == top ? 1.f : expf(from_key(key) - from_key(top));
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

template <int V>
__device__ __forceinline__ uint32_t local_max(const uint32_t (&key)[V])
{
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) m = max(m, key[v]);
    return m;
}

template <int L, int V, bool F32, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteParams p)
{
    extern __shared__ float stage[];      // per warp: [tokens][k] weights, then [tokens][k] experts
    constexpr int kTok = 32 / L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & (L - 1), tok = lane / L;
    const long long t0 = (static_cast<long long>(blockIdx.x) * kWarps + warp) * kTok;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (t0 >= p.T) return;
    float* sw = stage + warp * (2 * kTok * p.k);
    int* si = reinterpret_cast<int*>(sw + kTok * p.k);
    const bool live = t0 + tok < p.T;
    const long long base = (t0 + (live ? tok : 0)) * p.ld + sub * V;
    const int left = p.E - sub * V;       // elements of this lane
    uint32_t key[V];
    if constexpr (VEC) {
        constexpr int kPer = F32 ? 4 : 8;
#pragma unroll
        for (int c = 0; c < V / kPer; ++c) {
            uint4 u = make_uint4(0, 0, 0, 0);
            const bool in = c * kPer < left;
            if (in) u = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.logits) + base * (F32 ? 4 : 2)) + c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (F32) {
                    key[c * 4 + i] = in ? to_key(__uint_as_float(w[i])) : 0;
                } else {
                    key[c * 8 + 2 * i] = in ? to_key(__uint_as_float(w[i] << 16)) : 0;
                    key[c * 8 + 2 * i + 1] = in ? to_key(__uint_as_float(w[i] & 0xffff0000u)) : 0;
                }
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            key[v] = 0;
            if (v < left)
                key[v] = to_key(F32 ? __ldg(static_cast<const float*>(p.logits) + base + v)
                                    : __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[base + v]));
        }
    }
    uint32_t mine = local_max(key);
    const uint32_t top = group_max<L>(mine);
    float total = 0.f;
    if (!p.renormalize) {
#pragma unroll
        for (int v = 0; v < V; ++v) total += weight_of(key[v], top);
#pragma unroll
        for (int d = L / 2; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    }
    uint32_t best = top;
    for (int j = 0; j < p.k; ++j) {
        if (j) best = group_max<L>(mine);
        const float w = weight_of(best, top);
        if (p.renormalize) total += w;
        uint32_t who = __ballot_sync(0xffffffffu, mine == best);
        if (L < 32) who = (who >> (tok * L)) & ((1u << (L & 31)) - 1u);
        if (best == 0) {
            if (sub == 0) {
                sw[tok * p.k + j] = 0.f;
                si[tok * p.k + j] = -1;
            }
        } else if (sub == __ffs(who) - 1) {
            int at = -1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool hit = at < 0 && key[v] == best;
                at = hit ? v : at;
                key[v] = hit ? 0 : key[v];
            }
            mine = local_max(key);
            sw[tok * p.k + j] = w;
            si[tok * p.k + j] = sub * V + at;
        }
    }
    __syncwarp();
    const float inv = 1.f / total;        // infinite only where every weight is 0 and none is scaled
    const int n = static_cast<int>(min(static_cast<long long>(kTok), p.T - t0)) * p.k;
    for (int i = lane; i < (kTok * p.k + 31) / 32 * 32; i += 32) {
        const int tk = min(i / p.k, kTok - 1);
        const float f = __shfl_sync(0xffffffffu, inv, tk * L);
        if (i < n) {
            const float w = sw[i];
            p.gate_w[t0 * p.k + i] = w > 0.f ? w * f : 0.f;
            p.topk[t0 * p.k + i] = si[i];
        }
    }
}

template <int L, int V>
cudaError_t launch(const RouteParams& p, cudaStream_t stream, bool pdl)
{
    constexpr int kTok = 32 / L;
    const int es = p.f32 ? 4 : 2;
    const bool vec = p.E % (16 / es) == 0 && p.ld % (16 / es) == 0 && (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((p.T + kWarps * kTok - 1) / (kWarps * kTok));
    lc.blockDim = dim3(kWarps * 32);
    lc.dynamicSmemBytes = kWarps * kTok * p.k * 8;
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
