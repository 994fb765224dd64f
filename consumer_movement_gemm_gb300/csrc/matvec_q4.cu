// matvec_q4.cu -- up to 64 rows times a matrix of 4-bit weights with group
// scales, and the quantiser that lays such a matrix out.
//
//   out[t][n] = sum_g scale[g][n] * sum_{k in g} xs[t][k / 128] * x[t][k] * (nibble[k][n] - zero[g][n])
//
// Products of bf16 (or e4m3, exact in bf16) activations with the integers
// nibble - zero are exact, a group's sum is fp32, and the scales multiply it
// in fp32: nothing is rounded before the result.  The stream of weight blocks
// and the split are skinny.cuh's; rows beyond 32 go through the weights a
// second time, right behind the first (they come from L2 then).
#include "launch.cuh"
#include "skinny.cuh"

namespace tovl {

namespace {

using namespace skinny;
constexpr int kCta = skinny::kThreads;
constexpr int kPassRows = 32;
constexpr int kPartFloats = kPassRows * kCols;

constexpr int smem_size() { return base_smem(true) + 16; }

template <bool XS>
struct Worker {
    const MatvecParams& p;
    float* red;
    Ring<true> ring;
    int warp, lane;
    uint64_t pol;
    // blocks to fetch: position inside the (pass, k) blocks of tile f_tile
    int f_left, f_i, f_tile;

    __device__ __forceinline__ void fetch(int kb, int len)
    {
        if (f_left <= 0) return;
        if (lane == 0) ring.issue(p.w, f_tile * kCols, (f_i % kb) * kRowsQ4, 0, p.group, p.has_zero, pol);
        ring.filled();
        --f_left;
        f_i += kWarps;
        while (f_i >= len) {
            f_i -= len;
            ++f_tile;
        }
    }

    // The warp's share of blocks [.., i1) of a pass over rows r0 .. r0 + cnt.
    template <int NT>
    __device__ __forceinline__ void pass(int first, int i1, int r0, int cnt, int tile, float* part, int kb, int len)
    {
        const int g = lane >> 2, t = lane & 3;
        float acc[4][NT][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
        const int n_xs = (p.K + kXScaleGroup - 1) / kXScaleGroup;
        for (int i = first; i < i1; i += kWarps) {
            uint4 b[4][NT];
            float2 sx[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // a row past the last one repeats the first; its column is never stored
                const long long r = r0 + (nt * 8 + g < cnt ? nt * 8 + g : 0);
#pragma unroll
                for (int R = 0; R < 4; ++R) {
                    const int k = i * kRowsQ4 + 32 * R + 8 * t;
                    if (k >= p.K) {
                        b[R][nt] = make_uint4(0, 0, 0, 0);
                    } else if (XS) {
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x) + r * p.ldx + k));
                        const uint2 lo = e4m3x4_to_bf16(v.x), hi = e4m3x4_to_bf16(v.y);
                        b[R][nt] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    } else {
                        b[R][nt] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + r * p.ldx + k));
                    }
                }
                if (XS) {   // accumulator columns 2t and 2t + 1
                    const int c0 = nt * 8 + 2 * t;
                    sx[nt].x = c0 < cnt ? __ldg(p.x_scale + static_cast<long long>(r0 + c0) * n_xs + i) : 0.f;
                    sx[nt].y = c0 + 1 < cnt ? __ldg(p.x_scale + static_cast<long long>(r0 + c0 + 1) * n_xs + i) : 0.f;
                }
            }
            ring.wait(p.ctrl, p.pipe_timeout_ns);
            block_q4<NT, false, XS>(acc, b, b, sx, ring.stage(), ring.stage_meta(), p.group / 32, p.has_zero, lane);
            ring.taken();
            __syncwarp();      // every lane has read the stage before it is filled again
            fetch(kb, len);
        }
        const int col = threadIdx.x & 63, q = threadIdx.x >> 6;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt * 8 >= cnt) break;
            store_red<true, NT>(red, acc, nt, warp, lane);
            __syncthreads();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = q + 4 * u, row = nt * 8 + r;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += red[(w * 8 + r) * kRedPitch + col];
                if (row < cnt) {
                    if (part) part[row * kCols + col] = v;
                    else if (tile * kCols + col < p.N)
                        static_cast<__nv_bfloat16*>(p.out)[(r0 + row) * p.ldo + tile * kCols + col] = __float2bfloat16(v);
                }
            }
            __syncthreads();
        }
    }
};

template <bool XS>
__global__ void __launch_bounds__(kCta, 1) matvec_q4_kernel(const __grid_constant__ MatvecParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    float* red = reinterpret_cast<float*>(smem + ring_bytes(true) + meta_bytes(true));
    int* flag = reinterpret_cast<int*>(smem + base_smem(true) - 1024);
    Worker<XS> w{p, red};
    w.warp = threadIdx.x >> 5;
    w.lane = threadIdx.x & 31;
    w.pol = ptx::l2_policy(0);
    w.ring.init(smem, w.warp);
    if (w.lane == 0) {
        w.ring.init_barriers();
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.w.w);
        ptx::prefetch_tmap(&p.w.scale);
    }
    const int grid = gridDim.x, cta = blockIdx.x;
    const int kb = (p.K + kRowsQ4 - 1) / kRowsQ4;
    const int passes = (p.T + kPassRows - 1) / kPassRows;
    const int len = passes * kb, tiles = (p.N + kCols - 1) / kCols;
    const int total = tiles * len, per = blocks_per_cta(total, grid);
    const int b0 = min(cta * per, total), e0 = min(b0 + per, total);
    const int s0 = b0 + w.warp;
    w.f_left = e0 > s0 ? (e0 - s0 + kWarps - 1) / kWarps : 0;
    w.f_i = s0 % len;
    w.f_tile = s0 / len;
    __syncwarp();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
#pragma unroll 1
    for (int s = 0; s < Ring<true>::S; ++s) w.fetch(kb, len);

    for (int b = b0; b < e0;) {
        // (tile, pass): kb blocks, split where the CTA's range ends
        const int unit = b / kb, t0 = unit * kb, t1 = t0 + kb, end = min(t1, e0);
        const int tile = unit / passes, r0 = (unit % passes) * kPassRows;
        const int cnt = min(kPassRows, p.T - r0);
        const bool whole = b == t0 && end == t1;
        float* part = whole ? nullptr : p.part + (static_cast<long long>(cta) * 2 + (b == b0 ? 0 : 1)) * kPartFloats;
        const int first = b - t0 + ((w.warp - (b - b0)) & (kWarps - 1));
        if (cnt <= 8) w.template pass<1>(first, end - t0, r0, cnt, tile, part, kb, len);
        else if (cnt <= 16) w.template pass<2>(first, end - t0, r0, cnt, tile, part, kb, len);
        else w.template pass<4>(first, end - t0, r0, cnt, tile, part, kb, len);
        if (!whole) {
            const int c0 = t0 / per, c1 = (t1 - 1) / per;
            if (last_arrival(p.sync + c0, c1 - c0 + 1, flag)) {
                const int col = threadIdx.x & 63;
                if (tile * kCols + col < p.N) {
                    for (int r = threadIdx.x >> 6; r < cnt; r += kCta / kCols) {
                        float v = 0.f;
                        for (int k = c0; k <= c1; ++k)
                            v += __ldcg(p.part + (static_cast<long long>(k) * 2 + (t0 <= k * per ? 0 : 1)) * kPartFloats +
                                        r * kCols + col);
                        static_cast<__nv_bfloat16*>(p.out)[(r0 + r) * p.ldo + tile * kCols + col] = __float2bfloat16(v);
                    }
                }
            }
        }
        b = end;
    }
}

// One thread per column and group: the group's range gives scale and zero,
// then eight rows at a time become a word.  Reads the group twice (the second
// time from L1 / L2); runs once per weight matrix.
//
//   symmetric   scale = bf16(amax / 7),         nibble = 8 + round(w / scale), zero 8
//   with zeros  scale = bf16((max - min) / 15), zero = round(-min / scale), min <= 0 <= max
__global__ void __launch_bounds__(256) quantize_q4_kernel(const QuantParams p)
{
    ptx::grid_dep_wait();
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= p.N) return;
    const long long eg = blockIdx.y + static_cast<long long>(blockIdx.z) * gridDim.y;   // expert * groups + group
    const long long groups = p.K / p.group;
    if (eg >= groups * p.E) return;
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.w) + eg * p.group * p.N + n;
    float lo = 0.f, hi = 0.f;
    for (int i = 0; i < p.group; ++i) {
        const float v = __bfloat162float(w[static_cast<long long>(i) * p.N]);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    // the scale that the products use is the rounded one
    const float want = p.zero ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
    __nv_bfloat16 sb = __float2bfloat16(want);
    if (__bfloat162float(sb) < 1e-30f) sb = __float2bfloat16(1.f);    // a group of zeros
    const float s = __bfloat162float(sb);
    const int z = p.zero ? min(15, max(0, __float2int_rn(-lo / s))) : 8;
    static_cast<__nv_bfloat16*>(p.scale)[eg * p.N + n] = sb;
    if (p.zero) p.zero[eg * p.N + n] = static_cast<uint8_t>(z);
    for (int i = 0; i < p.group; i += 8) {
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = __bfloat162float(w[static_cast<long long>(i + j) * p.N]) / s;
            const int nib = min(15, max(0, __float2int_rn(fminf(fmaxf(v, -64.f), 64.f)) + z));
            word |= static_cast<uint32_t>(nib) << (4 * (j / 2) + 16 * (j & 1));
        }
        p.q[(eg * (p.group / 8) + i / 8) * p.N + n] = word;
    }
}

}  // namespace

cudaError_t prepare_matvec_q4()
{
    cudaError_t e = cudaFuncSetAttribute(matvec_q4_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_size());
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(matvec_q4_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_size());
    return e;
}

cudaError_t launch_matvec_q4(const MatvecParams& p, bool e4m3, int grid, cudaStream_t stream, bool pdl)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(kCta);
    lc.dynamicSmemBytes = smem_size();
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = pdl ? 1 : 0;
    return e4m3 ? cudaLaunchKernelEx(&lc, matvec_q4_kernel<true>, p) : cudaLaunchKernelEx(&lc, matvec_q4_kernel<false>, p);
}

cudaError_t launch_quantize_q4(const QuantParams& p, cudaStream_t stream)
{
    const long long eg = static_cast<long long>(p.K / p.group) * p.E;
    const unsigned y = eg < 32768 ? static_cast<unsigned>(eg) : 32768u;
    const unsigned z = static_cast<unsigned>((eg + y - 1) / y);
    quantize_q4_kernel<<<dim3((p.N + 255) / 256, y, z), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace tovl
