// rope_append.cu -- rotary embedding of a step's queries and keys, new keys and
// values written to their cache slots.
//
// A row is one head of one token; L threads (a power of two) share it, 16
// columns each as two pieces of 8: the two halves of eight rotated pairs, or
// neighbours where nothing is rotated.  So a thread has both numbers of every
// pair and eight cosines and sines, which it keeps for several heads of the same
// token.  Pairs are (i, i + rot/2), or (2 i, 2 i + 1) where they are
// interleaved.  Arithmetic is fp32, rounded once to bf16, or, for an e4m3 cache,
// to e4m3(x / scale) with scale = max(max |x|, 1e-12) / 448 of the row.
//
// What bounds it: a launch and dependent loads (position, slot, table) for few
// tokens; HBM for many.
#include <cuda_bf16.h>
#include "common.cuh"
#include "paged.cuh"
#include "sync.cuh"

namespace tovl {

namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                      ptx::pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// a, b: the pieces of one thread.  Interleaved pairs lie inside a piece.
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8], bool interleaved)
{
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], u = b[2 * i], w = b[2 * i + 1];
            a[2 * i] = x * c[i] - y * s[i], a[2 * i + 1] = y * c[i] + x * s[i];
            b[2 * i] = u * c[4 + i] - w * s[4 + i], b[2 * i + 1] = w * c[4 + i] + u * s[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * c[i] - y * s[i], b[i] = y * c[i] + x * s[i];
        }
    }
}

template <bool E4M3, int N>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p, int lanes, int units)
{
    const KvCache& cache = p.cache;
    const int D = cache.dim, rows = p.Hq + 2 * cache.heads;
    const int j = threadIdx.x & (lanes - 1);
    const long long u = (static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x) / lanes;
    const long long t = u / units;
    const int r0 = static_cast<int>(u - t * units) * N;
    const bool on = t < p.T;
    const bool turned = j < p.rot / 16;
    // pieces of 8 columns
    const int a = turned ? (p.interleaved ? 2 * j : j) : 2 * j;
    const int b = turned && !p.interleaved ? j + p.rot / 16 : a + 1;
    const bool has_a = a < D / 8, has_b = b < D / 8;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    uint4 xa[N], xb[N];
    int pos = 0, slot = -1;
    if (on) {
        pos = __ldg(p.positions + t);
        slot = __ldg(p.slots + t);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = r0 + i;
        xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
        if (!on || r >= rows) continue;
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(r < p.Hq ? p.q : r < p.Hq + cache.heads ? p.k : p.v);
        const int h = r < p.Hq ? r : r < p.Hq + cache.heads ? r - p.Hq : r - p.Hq - cache.heads;
        x += t * (r < p.Hq ? p.ldq : r < p.Hq + cache.heads ? p.ldk : p.ldv) + static_cast<long long>(h) * D;
        if (has_a) xa[i] = *reinterpret_cast<const uint4*>(x + a * 8);
        if (has_b) xb[i] = *reinterpret_cast<const uint4*>(x + b * 8);
    }
    bool write = on && slot >= 0;
    if (on && (slot < -1 || slot >= cache.pages * cache.page || (p.rot && slot >= 0 && (pos < 0 || pos >= p.max_pos)))) {
        record_error(p.ctrl, kErrInvalid);
        write = false;
    }
    float c[8], s[8];
    if (turned && on) {
        const float* at = p.cos_sin + static_cast<long long>(min(max(pos, 0), p.max_pos - 1)) * p.rot + 8 * j;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(at + i)), w = __ldg(reinterpret_cast<const float4*>(at + p.rot / 2 + i));
            c[i] = v.x, c[i + 1] = v.y, c[i + 2] = v.z, c[i + 3] = v.w;
            s[i] = w.x, s[i + 1] = w.y, s[i + 2] = w.z, s[i + 3] = w.w;
        }
    }
    const int page = !write ? 0 : cache.page_shift >= 0 ? slot >> cache.page_shift : slot / cache.page;
    const int in = write ? slot - page * cache.page : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = r0 + i;
        const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + cache.heads;
        const int h = is_q ? r : is_k ? r - p.Hq : r - p.Hq - cache.heads;
        const bool live = on && r < rows;
        float fa[8], fb[8];
        unpack8(xa[i], fa);
        unpack8(xb[i], fb);
        if (turned && live && (is_q || is_k)) rotate(fa, fb, c, s, p.interleaved);
        float inv = 0.f;
        if constexpr (E4M3) {
            // the largest magnitude by its bits, which put NaN on top
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, max(__float_as_uint(fa[k]) & 0x7fffffffu, __float_as_uint(fb[k]) & 0x7fffffffu));
            for (int d = 1; d < lanes; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float m = __uint_as_float(top);
            inv = (m < 1e-12f ? 1e-12f : m) / 448.f;
        }
        if (!live) continue;
        if (is_q) {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.q_out) + t * p.ldqo + static_cast<long long>(h) * D;
            if (has_a) *reinterpret_cast<uint4*>(o + a * 8) = pack8(fa);
            if (has_b) *reinterpret_cast<uint4*>(o + b * 8) = pack8(fb);
        } else if (write) {
            uint8_t* o = (is_k ? cache.k : cache.v) + page * cache.page_stride + in * cache.slot_stride + h * cache.head_stride;
            if constexpr (E4M3) {
                const auto eight = [&](const float (&x)[8]) {
                    const float y[8] = {x[0] / inv, x[1] / inv, x[2] / inv, x[3] / inv, x[4] / inv, x[5] / inv, x[6] / inv, x[7] / inv};
                    return make_uint2(to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16, to_e4m3x2(y[4], y[5]) | to_e4m3x2(y[6], y[7]) << 16);
                };
                if (has_a) *reinterpret_cast<uint2*>(o + a * 8) = eight(fa);
                if (has_b) *reinterpret_cast<uint2*>(o + b * 8) = eight(fb);
                if (j == 0) (is_k ? cache.k_scale : cache.v_scale)[(static_cast<long long>(page) * cache.heads + h) * cache.page + in] = inv;
            } else {
                if (has_a) *reinterpret_cast<uint4*>(o + a * 16) = pack8(fa);
                if (has_b) *reinterpret_cast<uint4*>(o + b * 16) = pack8(fb);
            }
        }
    }
}

template <int N>
cudaError_t launch(const RopeParams& p, bool e4m3, cudaStream_t stream, bool pdl)
{
    int lanes = 1;
    while (lanes * 16 < p.cache.dim) lanes *= 2;
    const int units = (p.Hq + 2 * p.cache.heads + N - 1) / N;
    const long long threads = static_cast<long long>(p.T) * units * lanes;
    const long long grid = (threads + kRopeThreads - 1) / kRopeThreads;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(grid));
    lc.blockDim = dim3(kRopeThreads);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = pdl ? 1 : 0;
    return e4m3 ? cudaLaunchKernelEx(&lc, rope_append_kernel<true, N>, p, lanes, units)
                : cudaLaunchKernelEx(&lc, rope_append_kernel<false, N>, p, lanes, units);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, bool e4m3, int num_sms, cudaStream_t stream, bool pdl)
{
    // four heads a thread where that leaves several CTAs for every SM
    const long long rows = static_cast<long long>(p.T) * (p.Hq + 2 * p.cache.heads);
    return rows * p.cache.dim / 16 >= 8LL * kRopeThreads * num_sms * 4 ? launch<4>(p, e4m3, stream, pdl) : launch<1>(p, e4m3, stream, pdl);
}

}  // namespace tovl
