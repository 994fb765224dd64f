// rope_append.cu -- rotary embedding of a step's queries and keys, new keys and
// values written to their cache slots.
//
// A row is one head of one token; ceil(dim / 16) lanes share it, 16 columns each
// as two pieces of 8, half of what is rotated (or is not) apart, so that a warp's
// accesses are whole lines.  So a lane has both numbers of every pair, (i, i +
// rot/2) or interleaved (2 i, 2 i + 1), and eight cosines and sines, which it keeps
// for one or three heads of its token; a CTA has one token.  Arithmetic is fp32,
// rounded once to bf16, or, for an e4m3 cache, to e4m3(x / scale) with scale =
// max(max |x|, 1e-12) / 448 of the row.
//
// What bounds it: a launch and dependent loads (position, slot, angles) for few
// tokens (1 token, 32 + 2 x 8 heads of 128: 1.7 us); HBM for many (16384 tokens
// 67 us, 6.1 TB/s, with 24 warps an SM, whose 64 registers leave 28 bytes a thread in
// local memory where a lane has three heads; 72 us with the 22 warps of unlimited ones).
#include <cuda_bf16.h>
#include "common.cuh"
#include "paged.cuh"
#include "sync.cuh"

namespace tovl {

namespace {

constexpr int kMostWarps = 8;          // of a CTA

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

// The quotients of a row by its scale, taken to 2^-46 by one residual before their
// own rounding (Markstein 1990): a product with the inverse alone would round
// twice, and miss ties.  16384 tokens, 32 + 2 x 8 heads of 128: 76 us, with the
// product alone 73, with a division 88.
struct Scale {
    float s, inverse;
    __device__ __forceinline__ explicit Scale(float top) : s((top < 1e-12f ? 1e-12f : top) / 448.f), inverse(1.f / s) {}
    __device__ __forceinline__ float divide(float x) const
    {
        const float q = x * inverse;
        return fmaf(fmaf(-q, s == INFINITY ? 0.f : s, x), inverse, q);
    }
};

__device__ __forceinline__ uint2 to_e4m3x8(const float (&x)[8], const Scale& s)
{
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = to_e4m3x2(s.divide(x[2 * i]), s.divide(x[2 * i + 1]));
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// lanes: of a row; units: groups of N rows of a token
template <bool E4M3, int N>
__global__ void __maxnreg__(64) rope_append_kernel(const RopeParams p, int lanes, int units)
{
    const KvCache& cache = p.cache;
    const int D = cache.dim, rows = p.Hq + 2 * cache.heads, lane = threadIdx.x & 31;
    const int per_warp = 32 / lanes, mine = lane / lanes, j = lane - mine * lanes;
    const int unit = ((blockIdx.y * blockDim.x + threadIdx.x) / 32) * per_warp + mine;
    const long long t = blockIdx.x;
    const int r0 = unit * N;
    const bool on = mine < per_warp && unit < units;
    const bool turned = j < p.rot / 16;
    // pieces of 8 columns: the halves of what is rotated, then those of the rest
    const int half = turned ? p.rot / 16 : (D / 8 - p.rot / 8 + 1) / 2;
    const int a = turned ? j : p.rot / 8 + j - p.rot / 16, b = a + half;
    const bool has_a = turned || j - p.rot / 16 < half, has_b = has_a && b < D / 8;
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
        // angles of the pairs (a's first and b's first column, ..), or of a's four and of b's four
        const float* at = p.cos_sin + static_cast<long long>(min(max(pos, 0), p.max_pos - 1)) * p.rot;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float* pairs = at + (!p.interleaved ? 8 * j + i : 4 * (i ? b : a));
            const float4 v = __ldg(reinterpret_cast<const float4*>(pairs)), w = __ldg(reinterpret_cast<const float4*>(pairs + p.rot / 2));
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
        uint32_t top = 0;
        if (E4M3 && __any_sync(0xffffffffu, live && !is_q)) {
            // the row's largest magnitude by its bits, which put NaN on top
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, max(__float_as_uint(fa[k]) & 0x7fffffffu, __float_as_uint(fb[k]) & 0x7fffffffu));
            for (int d = 1; d < lanes; d *= 2) {
                const uint32_t o = __shfl_down_sync(0xffffffffu, top, d);
                if (j + d < lanes) top = max(top, o);
            }
            top = __shfl_sync(0xffffffffu, top, lane - j);
        }
        if (!live) continue;
        if (is_q) {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.q_out) + t * p.ldqo + static_cast<long long>(h) * D;
            if (has_a) *reinterpret_cast<uint4*>(o + a * 8) = pack8(fa);
            if (has_b) *reinterpret_cast<uint4*>(o + b * 8) = pack8(fb);
        } else if (write) {
            uint8_t* o = (is_k ? cache.k : cache.v) + page * cache.page_stride + in * cache.slot_stride + h * cache.head_stride;
            if constexpr (E4M3) {
                const Scale scale(__uint_as_float(top));
                if (has_a) *reinterpret_cast<uint2*>(o + a * 8) = to_e4m3x8(fa, scale);
                if (has_b) *reinterpret_cast<uint2*>(o + b * 8) = to_e4m3x8(fb, scale);
                if (j == 0) (is_k ? cache.k_scale : cache.v_scale)[(static_cast<long long>(page) * cache.heads + h) * cache.page + in] = scale.s;
            } else {
                if (has_a) *reinterpret_cast<uint4*>(o + a * 16) = pack8(fa);
                if (has_b) *reinterpret_cast<uint4*>(o + b * 16) = pack8(fb);
            }
        }
    }
}

template <int N>
cudaError_t launch(const RopeParams& p, bool e4m3, int lanes, cudaStream_t stream, bool pdl)
{
    const int units = (p.Hq + 2 * p.cache.heads + N - 1) / N, warps = (units + 32 / lanes - 1) / (32 / lanes);
    const int blocks = (warps + kMostWarps - 1) / kMostWarps;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(p.T), static_cast<unsigned>(blocks));
    lc.blockDim = dim3(static_cast<unsigned>((warps + blocks - 1) / blocks) * 32);
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
    const int lanes = (p.cache.dim + 15) / 16;
    // three heads a lane where that leaves eight warps for every SM.  16384 tokens, 32 +
    // 2 x 8 heads, three / four, us: of 128 67.4 / 68.8 (two 74), of 64 35.3 / 37.9, of 80
    // 49.7 / 51.3, of 256 (8 + 2 x 2) 35.7 / 38.4; e4m3, of 64 48 / 58, of 80 62 / 69, of 96
    // 72 / 79, of 256 48 / 57, of 192 (16 + 2 x 4) 71 / 71, of 128 75.8 / 72.3 and (64 + 2 x 8)
    // 134 / 120: only there are four better.  Up to 256 tokens one head is as good.
    const long long warps = static_cast<long long>(p.T) * (p.Hq + 2 * p.cache.heads) * lanes / 32;
    return warps < 32LL * num_sms ? launch<1>(p, e4m3, lanes, stream, pdl) : launch<3>(p, e4m3, lanes, stream, pdl);
}

}  // namespace tovl
