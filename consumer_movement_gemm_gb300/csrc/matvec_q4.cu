// matvec_q4.cu -- up to 64 rows times a matrix of 4-bit weights with group
// scales, and the quantiser that lays such a matrix out.
//
//   out[t][n] = sum_g scale[g][n] * sum_{k in g} xs[t][k / 128] * x[t][k] * (nibble[k][n] - zero[g][n])
//
// The activations enter the tensor core as fp16 (e4m3 exactly, bf16 with a
// power of two per 128 columns), their products with the integers nibble -
// zero are exact, a group's sum is fp32, and the scales multiply it in fp32:
// nothing is rounded before the result.  Every 16 rows are a pass over
// the weights (fp16 rows and their sums, two 8-row tiles of the instruction, are
// what the registers hold), a pass the next one's matrix, so large matrices are
// read again.
//
// Large products stream the weights through skinny.cuh's rings, small ones read
// them straight into registers (matvec_q4_direct.cuh); use_direct is the rule.
// What bounds the ring: instruction issue, about 400 instructions per 2 KB of
// weights with 9 to 16 rows and 335 with up to 8.  16 x 7168 x 32768: 43.7 us, 2.8
// TB/s; 1 x 8192 x 28672: 30.4 us, 4.0 TB/s.
#include <type_traits>
#include "launch.cuh"
#include "matvec_q4_direct.cuh"
#include "skinny.cuh"

namespace tovl {

namespace {

using namespace skinny;
constexpr int kPassRows = 16;
constexpr int kThreads4 = Shape<128>::kThreads;

struct Tables {
    Product pr;
    int last;
    Queue queue;
};

template <int G>
constexpr int smem_size() { return 1024 + Shape<G>::kRing + kRowBuffers + static_cast<int>(sizeof(Tables)) + 16; }

struct Calls {
    const MatvecParams& p;
    __device__ __forceinline__ const WeightMaps* maps(int) const { return &p.w; }
    __device__ __forceinline__ int expert(int, int) const { return 0; }
};

// A segment of a pass over rows r0 .. r0 + cnt.
template <int NT, bool XS, int G, bool Z>
__device__ __forceinline__ void run_segment(const MatvecParams& p, Engine<G, Z, Calls>& eng, int r0, int cnt, int tile, int i0,
                                            int i1, int number)
{
    const int n_xs = (p.K + kXScaleGroup - 1) / kXScaleGroup;
    float* part = p.part + (static_cast<long long>(number) * p.T + r0) * p.N;
    eng.template segment<NT, XS ? Rows::kE4m3 : Rows::kBf16>(
        i0, i1, part, p.N, cnt, tile * kTileCols, p.N, p.K,
        [&](int r, int k, bool) {
            const long long at = (r0 + r) * p.ldx + k;
            if (!XS) return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + at));
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x) + at));
            return make_uint4(v.x, v.y, 0, 0);
        },
        [&](int r, int k) { return __ldg(p.x_scale + static_cast<long long>(r0 + r) * n_xs + k / kXScaleGroup); });
}

template <bool XS, int G, bool Z>
__global__ void __launch_bounds__(Shape<G>::kThreads, 1) matvec_q4_kernel(const __grid_constant__ MatvecParams p)
{
    using P = Shape<G>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    uint8_t* rows_buf = smem + (P::kRing + 15) / 16 * 16;
    Tables& tb = *reinterpret_cast<Tables*>(rows_buf + kRowBuffers);
    const Calls calls{p};
    Engine<G, Z, Calls> eng{calls, &tb.pr, &tb.queue, p.sync + kTicketWord, p.ctrl, p.pipe_timeout_ns, 1};
    eng.warp = threadIdx.x >> 5;
    eng.lane = threadIdx.x & 31;
    eng.init(smem, rows_buf);
    if (threadIdx.x == 0) {
        ptx::prefetch_tmap(&p.w.w);
        ptx::prefetch_tmap(&p.w.scale);
    }
    const int grid = gridDim.x;
    const int passes = (p.T + kPassRows - 1) / kPassRows;      // as matrices of the product
    if (threadIdx.x == 0) tb.pr.init(passes, p.N, p.K, P::kRows, P::kUnitBytes, grid, p.most_parts);
    for (int i = threadIdx.x; i < kMaxItems + 8; i += P::kThreads) tb.queue.item[i] = kNoItem;
    __syncthreads();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    eng.start();
    eng.walk(0, [&](int matrix, int tile, int i0, int i1, int number) {
        const int r0 = matrix * kPassRows, cnt = min(kPassRows, p.T - r0);
        if (cnt <= 8) run_segment<1, XS, G, Z>(p, eng, r0, cnt, tile, i0, i1, number);
        else run_segment<2, XS, G, Z>(p, eng, r0, cnt, tile, i0, i1, number);
        // the last CTA to finish a part of the tile adds them all (no CTA
        // waits for another one, so none has to be resident)
        const int t0 = (matrix * tb.pr.tiles + tile) * tb.pr.kb, parts = tb.pr.parts(t0);
        __syncthreads();
        if (parts > 1) {
            if (threadIdx.x == 0) {
                int* counter = p.sync + kPartWord + tb.pr.item_of(t0);
                const bool last = ptx::atom_add_acq_rel_gpu(counter, 1) == parts - 1;
                if (last) ptx::st_relaxed_gpu(counter, 0);
                tb.last = last;
            }
            __syncthreads();
            if (!tb.last) return;
        }
        const int quads = min(kTileCols, p.N - tile * kTileCols) / 4;
        for (int i = threadIdx.x; i < cnt * quads; i += P::kThreads) {
            const int r = i / quads, n = tile * kTileCols + (i - r * quads) * 4;
            const float* const part[1] = {p.part + static_cast<long long>(r0 + r) * p.N + n};
            const int count[1] = {parts};
            float4 s[1];
            add_parts<1>(s, part, count, static_cast<long long>(p.T) * p.N);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (r0 + r) * p.ldo + n;
            if (p.out_vec) {
                *reinterpret_cast<uint2*>(out) = make_uint2(ptx::pack_bf16x2(s[0].x, s[0].y), ptx::pack_bf16x2(s[0].z, s[0].w));
            } else {
                out[0] = __float2bfloat16(s[0].x), out[1] = __float2bfloat16(s[0].y);
                out[2] = __float2bfloat16(s[0].z), out[3] = __float2bfloat16(s[0].w);
            }
        }
    });
    // the last CTA to leave clears the tickets for the next call
    if (tb.pr.tickets && threadIdx.x == 0 && ptx::atom_add_relaxed_gpu(p.sync + kExitWord, 1) == grid - 1) {
        ptx::st_relaxed_gpu(p.sync + kTicketWord, 0);
        ptx::st_relaxed_gpu(p.sync + kExitWord, 0);
    }
}

// One thread per column and group: the group's range gives scale and zero,
// then eight rows at a time become a word.  Reads the group twice (the second
// time from L1 / L2); runs once per weight matrix.  8192 x 28672: 319 us, bound by
// a division and its rounding per weight (with the group in registers and one
// pass over memory, at half the warps, 380).
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
    // the scale that the products use is the rounded one (halves: hi - lo may be
    // over the largest number)
    const float want = p.zero ? (0.5f * hi - 0.5f * lo) / 7.5f : fmaxf(hi, -lo) / 7.f;
    __nv_bfloat16 sb = __float2bfloat16(want);
    if (__bfloat162float(sb) == 0.f) sb = __float2bfloat16(1.f);      // a group of zeros
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

// Calls f with the kernel of an activation type, group and zeros.
template <class F>
static cudaError_t with_kernel(bool e4m3, int group, bool zero, F f)
{
    const auto pick = [&](auto xs, auto g) {
        constexpr int G = decltype(g)::value;
        return zero ? f(matvec_q4_kernel<decltype(xs)::value, G, true>, smem_size<G>())
                    : f(matvec_q4_kernel<decltype(xs)::value, G, false>, smem_size<G>());
    };
    const auto by_group = [&](auto xs) {
        if (group == 32) return pick(xs, std::integral_constant<int, 32>());
        if (group == 64) return pick(xs, std::integral_constant<int, 64>());
        return pick(xs, std::integral_constant<int, 128>());
    };
    return e4m3 ? by_group(std::true_type()) : by_group(std::false_type());
}

cudaError_t prepare_matvec_q4()
{
    for (int i = 0; i < 12; ++i) {
        const cudaError_t e = with_kernel(i & 1, 32 << (i >> 2), (i >> 1) & 1, [](auto kernel, int smem) {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        });
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int NT, bool XS, int G>
static cudaError_t launch_direct(const MatvecDirectParams& p, bool zero, int sms, cudaStream_t stream, bool pdl)
{
    const int tiles = (p.N + kDirectCols - 1) / kDirectCols, passes = (p.T + 15) / 16, blocks = (p.K + 127) / 128;
    // One CTA of 16 warps per SM where that is all of them; else CTAs of 8, two
    // on an SM, whose starts and ends overlap (one row: 128 tiles, 11008 x 4096,
    // 9.9 us with 16 and 11.3 with 8; 344 tiles, 4096 x 11008, 12.5 and 11.1).
    // Clusters as long as they fit the SMs and leave each warp a block (28672 x
    // 1024: 20.9 us without, 8.2 with four CTAs; eight are no faster than four:
    // 28672 x 512 9.5 and 8.2).
    const int warps = tiles * passes <= sms ? kDirectWarps : kDirectWarps / 2;
    int split = 1;
    while (split < kDirectCluster && tiles * passes * split * 2 <= sms && split * warps < blocks) split *= 2;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(tiles, split, passes);
    lc.blockDim = dim3(warps * 32);
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (split > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 1;
        attr[n].val.clusterDim.y = split;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    lc.attrs = attr;
    lc.numAttrs = n;
    return zero ? cudaLaunchKernelEx(&lc, matvec_q4_direct_kernel<NT, XS, G, true>, p)
                : cudaLaunchKernelEx(&lc, matvec_q4_direct_kernel<NT, XS, G, false>, p);
}

template <int NT, bool XS>
static cudaError_t launch_direct(const MatvecDirectParams& p, int group, bool zero, int sms, cudaStream_t stream, bool pdl)
{
    if (group == 32) return launch_direct<NT, XS, 32>(p, zero, sms, stream, pdl);
    if (group == 64) return launch_direct<NT, XS, 64>(p, zero, sms, stream, pdl);
    return launch_direct<NT, XS, 128>(p, zero, sms, stream, pdl);
}

cudaError_t launch_matvec_q4_direct(const MatvecDirectParams& p, bool e4m3, int group, bool zero, int sms, cudaStream_t stream,
                                    bool pdl)
{
    if (p.T <= 8)
        return e4m3 ? launch_direct<1, true>(p, group, zero, sms, stream, pdl) : launch_direct<1, false>(p, group, zero, sms, stream, pdl);
    return e4m3 ? launch_direct<2, true>(p, group, zero, sms, stream, pdl) : launch_direct<2, false>(p, group, zero, sms, stream, pdl);
}

cudaError_t launch_matvec_q4(const MatvecParams& p, bool e4m3, int group, bool zero, int grid, cudaStream_t stream,
                             bool pdl)
{
    return with_kernel(e4m3, group, zero, [&](auto kernel, int smem) {
        return launch_grid(kernel, p, grid, kThreads4, smem, stream, false, pdl);
    });
}

cudaError_t launch_quantize_q4(const QuantParams& p, cudaStream_t stream)
{
    const long long eg = static_cast<long long>(p.K / p.group) * p.E;
    const unsigned y = eg < 32768 ? static_cast<unsigned>(eg) : 32768u;
    const unsigned z = static_cast<unsigned>((eg + y - 1) / y);
    quantize_q4_kernel<<<dim3((p.N - 1) / 256 + 1, y, z), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace tovl
