// moe_decode.cu -- a whole gated expert layer for up to 64 tokens in one kernel.
//
//   h[t, e]  = silu(x[t] W13[e][:, :I]) * (x[t] W13[e][:, I:])      for the experts e that token t names
//   out[t]   = sum over those e of gate[t, e] * (h[t, e] W2[e])
//
// One persistent grid, one CTA per SM, four steps with a grid barrier between
// them: the first product's parts, h (all CTAs add the parts and apply the
// activation), the second product's parts, out (added over parts and
// experts).  The two products run on one engine (skinny.cuh) whose rings of
// weight stages go straight on from W13 to W2: the memory system keeps
// delivering while the CTAs meet.  Only the experts that some token names are
// listed, each with the tokens that name it as its rows.
//
// Roundings: x and the weights are bf16 (or 4-bit with their scales applied
// in fp32), sums are fp32.  h is split into two bf16 numbers, its rounding
// and the rest, and the second product multiplies both (the second one rides
// on the same weight fragments): one bf16 h would raise the error of the
// result from its own rounding's 1.7e-3 to 2.4e-3, the pair leaves it alone.
#include <type_traits>
#include "launch.cuh"
#include "skinny.cuh"

namespace tovl {

namespace {

using namespace skinny;

constexpr int kMaxPairs = kMaxDecodeRows * kMaxDecodeK;
constexpr int kMaxEntries = kMaxExperts + kMaxPairs / 16;

// An expert, or the rows of one that a pass takes.
__device__ __forceinline__ uint32_t pack_entry(int e, int cnt, int off) { return e | (cnt - 1) << 10 | off << 16; }
__device__ __forceinline__ int entry_expert(uint32_t v) { return v & 1023; }
__device__ __forceinline__ int entry_rows(uint32_t v) { return ((v >> 10) & 63) + 1; }
__device__ __forceinline__ int entry_off(uint32_t v) { return v >> 16; }

struct Tables {
    Product pr[2];
    Queue queue[2];
    uint32_t entry[kMaxEntries];
    int16_t pair_row[kMaxPairs];            // row of each (token, slot); -1: no expert, or one that an earlier slot names
    float pair_w[kMaxPairs];                // its gate weight, with those of later slots that name the expert too
    uint16_t row_entry[kMaxPairs];
    uint8_t row_tok[kMaxPairs];
    int16_t topk[kMaxPairs];
    float gate[kMaxPairs];
    unsigned long long mask[kMaxExperts];   // tokens of each expert
    int n_entries, n_rows, bad;
};

template <int G>
constexpr int smem_size() { return 1024 + Shape<G>::kRing + kRowBuffers + static_cast<int>(sizeof(Tables)) + 16; }

// Builds the list of experts with rows.  Every CTA builds the same list
// (ascending experts, ascending tokens), so they agree on row numbers without
// talking.  A token that names an expert twice has one row with both weights.
// False if an id is outside [-1, E).
template <int PASS, int THREADS>
__device__ bool build_tables(const MoeParams& p, Tables& tb)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const int pairs = p.T * p.k;
    constexpr int kPer = (kMaxPairs + THREADS - 1) / THREADS;
    int id[kPer];
    float w[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int i = tid + u * THREADS;
        id[u] = i < pairs ? __ldg(p.topk + i) : -1;
        w[u] = i < pairs ? __ldg(p.gate_w + i) : 0.f;
    }
    for (int e = tid; e < p.E; e += THREADS) tb.mask[e] = 0;
    if (tid == 0) tb.bad = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int i = tid + u * THREADS;
        if (i < pairs) {
            if (id[u] < -1 || id[u] >= p.E) {
                tb.bad = 1;
                id[u] = -1;
            }
            tb.topk[i] = static_cast<int16_t>(id[u]);
            tb.gate[i] = w[u];
            if (id[u] >= 0) atomicOr(tb.mask + id[u], 1ull << (i / p.k));
        }
    }
    __syncthreads();
    if (tb.bad) return false;
    if (tid < 32) {
        int n = 0, rows = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            unsigned long long m = e < p.E ? tb.mask[e] : 0;
            const int cnt = __popcll(m), passes = (cnt + PASS - 1) / PASS;
            int sn = passes, sr = cnt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, sn, d), b = __shfl_up_sync(0xffffffffu, sr, d);
                if (lane >= d) {
                    sn += a;
                    sr += b;
                }
            }
            const int first = n + sn - passes, off = rows + sr - cnt;
            for (int q = 0; q < passes; ++q)
                tb.entry[first + q] = pack_entry(e, min(cnt - q * PASS, PASS), off + q * PASS);
            for (int r = 0; m; ++r, m &= m - 1) {
                tb.row_tok[off + r] = static_cast<uint8_t>(__ffsll(m) - 1);
                tb.row_entry[off + r] = static_cast<uint16_t>(first + r / PASS);
            }
            n += __shfl_sync(0xffffffffu, sn, 31);
            rows += __shfl_sync(0xffffffffu, sr, 31);
        }
        if (lane == 0) {
            tb.n_entries = n;
            tb.n_rows = rows;
        }
    }
    __syncthreads();
    return true;
}

// Row and weight of every (token, slot); read after the next barrier.
template <int THREADS>
__device__ void build_pairs(const MoeParams& p, Tables& tb)
{
    for (int i = threadIdx.x; i < p.T * p.k; i += THREADS) tb.pair_row[i] = -1;
    __syncthreads();
    for (int r = threadIdx.x; r < tb.n_rows; r += THREADS) {
        const int e = entry_expert(tb.entry[tb.row_entry[r]]), t = tb.row_tok[r];
        int first = -1;
        float w = 0.f;
        for (int j = 0; j < p.k; ++j)
            if (tb.topk[t * p.k + j] == e) {
                if (first < 0) first = j;
                w += tb.gate[t * p.k + j];
            }
        tb.pair_row[t * p.k + first] = static_cast<int16_t>(r);
        tb.pair_w[t * p.k + first] = w;
    }
}

struct Calls {
    const MoeParams& p;
    const Tables& tb;
    __device__ __forceinline__ const WeightMaps& maps(int ph) const { return ph ? p.w2 : p.w13; }
    __device__ __forceinline__ int expert(int, int matrix) const { return entry_expert(tb.entry[matrix]); }
};

template <int G, bool Z>
struct Worker {
    using P = Shape<G>;
    const MoeParams& p;
    const Tables& tb;
    Engine<G, Z, Calls>& eng;

    // A segment of a product with NT * 8 rows: x (H false) or h (H true).
    template <int NT, bool H>
    __device__ __forceinline__ void segment(uint32_t en, int tile, int i0, int i1, int number)
    {
        const int cnt = entry_rows(en), off = entry_off(en);
        const int K = H ? p.I : p.H, N = H ? p.H : 2 * p.I;
        float* part = p.part + (static_cast<long long>(number) * p.T * p.k + off) * N;
        eng.template segment<NT, H, false>(
            i0, i1, part, N, cnt, tile * kTileCols, N, K,
            [&](int r, int k, bool lo) {
                if (H) {     // (written in this launch)
                    const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(lo ? p.h_lo : p.h_hi);
                    return __ldcg(reinterpret_cast<const uint4*>(h + static_cast<long long>(off + r) * p.I + k));
                }
                return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + tb.row_tok[off + r] * p.ldx + k));
            },
            [](int, int) { return 1.f; });
    }

    template <bool H>
    __device__ __forceinline__ void product()
    {
        eng.walk(H, [&](int matrix, int tile, int i0, int i1, int number) {
            const uint32_t en = tb.entry[matrix];
            const int cnt = entry_rows(en);
            if (cnt <= 8) segment<1, H>(en, tile, i0, i1, number);
            else if (cnt <= 16) segment<2, H>(en, tile, i0, i1, number);
            else if (cnt <= 32) segment<4, H>(en, tile, i0, i1, number);
            else if constexpr (P::kPassRows > 32) segment<8, H>(en, tile, i0, i1, number);
        });
    }

    // Sum of the parts of four columns of a row of product `ph`.
    __device__ __forceinline__ float4 total(int ph, int row, int n, int N) const
    {
        const Product& q = tb.pr[ph];
        const int t0 = (tb.row_entry[row] * q.tiles + n / kTileCols) * q.kb;
        return add_parts(p.part + static_cast<long long>(row) * N + n, q.parts(t0), static_cast<long long>(p.T) * p.k * N);
    }

    __device__ __forceinline__ void activations()
    {
        const int quads = p.I / 4;
        for (int i = blockIdx.x * P::kThreads + threadIdx.x; i < tb.n_rows * quads; i += gridDim.x * P::kThreads) {
            const int row = i / quads, n = (i - row * quads) * 4;
            const float4 g4 = total(0, row, n, 2 * p.I), u4 = total(0, row, p.I + n, 2 * p.I);
            const float g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
            float hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float h = g[j] / (1.f + expf(-g[j])) * u[j];
                hi[j] = __bfloat162float(__float2bfloat16(h));
                // (an overflowed h has no second part)
                lo[j] = fabsf(h - hi[j]) < INFINITY ? h - hi[j] : 0.f;
            }
            const long long at = static_cast<long long>(row) * p.I + n;
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.h_hi) + at) =
                make_uint2(ptx::pack_bf16x2(hi[0], hi[1]), ptx::pack_bf16x2(hi[2], hi[3]));
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.h_lo) + at) =
                make_uint2(ptx::pack_bf16x2(lo[0], lo[1]), ptx::pack_bf16x2(lo[2], lo[3]));
        }
    }

    __device__ __forceinline__ void outputs()
    {
        const int quads = p.H / 4;
        for (int i = blockIdx.x * P::kThreads + threadIdx.x; i < p.T * quads; i += gridDim.x * P::kThreads) {
            const int t = i / quads, n = (i - t * quads) * 4;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j = 0; j < p.k; ++j) {
                const int row = tb.pair_row[t * p.k + j];
                if (row < 0) continue;
                const float w = tb.pair_w[t * p.k + j];
                const float4 v = total(1, row, n, p.H);
                s.x += w * v.x, s.y += w * v.y, s.z += w * v.z, s.w += w * v.w;
            }
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + t * p.ldo + n;
            const uint32_t lo = ptx::pack_bf16x2(s.x, s.y), hi = ptx::pack_bf16x2(s.z, s.w);
            if (p.out_vec) {
                *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
            } else {
                out[0] = __float2bfloat16(s.x), out[1] = __float2bfloat16(s.y);
                out[2] = __float2bfloat16(s.z), out[3] = __float2bfloat16(s.w);
            }
        }
    }
};

template <int G, bool Z>
__global__ void __launch_bounds__(Shape<G>::kThreads, 1) moe_decode_kernel(const __grid_constant__ MoeParams p)
{
    using P = Shape<G>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    uint8_t* rows_buf = smem + (P::kRing + 15) / 16 * 16;
    Tables& tb = *reinterpret_cast<Tables*>(rows_buf + kRowBuffers);
    const Calls calls{p, tb};
    Engine<G, Z, Calls> eng{calls, tb.pr, tb.queue, rows_buf, p.sync + kTicketWord, p.ctrl, p.pipe_timeout_ns, 2};
    eng.warp = threadIdx.x >> 5;
    eng.lane = threadIdx.x & 31;
    eng.ring.init(smem, eng.warp);
    if (eng.lane == 0) {
        eng.ring.init_barriers();
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.w13.w);
        ptx::prefetch_tmap(&p.w2.w);
    }
    for (int i = threadIdx.x; i < 2 * (kMaxItems + 8); i += P::kThreads)
        tb.queue[i / (kMaxItems + 8)].item[i % (kMaxItems + 8)] = kNoItem;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int grid = gridDim.x;
    if (!build_tables<P::kPassRows, P::kThreads>(p, tb)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_error(p.ctrl, kErrInvalid);
        return;
    }
    if (threadIdx.x < 2)
        tb.pr[threadIdx.x].init(tb.n_entries, threadIdx.x ? p.H : 2 * p.I, threadIdx.x ? p.I : p.H, P::kRows, grid, p.most_parts);
    __syncthreads();
    eng.start();
    build_pairs<P::kThreads>(p, tb);
    Worker<G, Z> w{p, tb, eng};
    w.template product<false>();
    grid_barrier(p.sync + kBarrierWord, grid + p.ready_offset, p.ctrl, p.timeout_ns);
    w.activations();
    grid_barrier(p.sync + kBarrierWord + 32, grid, p.ctrl, p.timeout_ns);
    w.template product<true>();
    grid_barrier(p.sync + kBarrierWord + 64, grid, p.ctrl, p.timeout_ns);
    w.outputs();
    // the last CTA past the last barrier clears the counters for the next call
    if (threadIdx.x == 0 && ptx::atom_add_relaxed_gpu(p.sync + kExitWord, 1) == grid - 1)
        for (int i = 0; i < kSyncWords; i += kSyncStep) ptx::st_relaxed_gpu(p.sync + i, 0);
}

}  // namespace

// Calls f with the kernel of a weight type, its threads and shared memory.
template <class F>
static cudaError_t with_kernel(int group, bool zero, F f)
{
    const auto zeros = [&](auto g) {
        constexpr int G = decltype(g)::value;
        return zero ? f(moe_decode_kernel<G, true>, Shape<G>::kThreads, smem_size<G>())
                    : f(moe_decode_kernel<G, false>, Shape<G>::kThreads, smem_size<G>());
    };
    switch (group) {
    case 32: return zeros(std::integral_constant<int, 32>());
    case 64: return zeros(std::integral_constant<int, 64>());
    case 128: return zeros(std::integral_constant<int, 128>());
    default: return f(moe_decode_kernel<0, false>, Shape<0>::kThreads, smem_size<0>());
    }
}

cudaError_t prepare_moe_decode()
{
    for (int group : {0, 32, 64, 128})
        for (bool zero : {false, true}) {
            const cudaError_t e = with_kernel(group, zero, [&](auto kernel, int, int smem) {
                return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            });
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t launch_moe_decode(const MoeParams& p, int group, bool zero, int grid, cudaStream_t stream, bool cooperative,
                              bool pdl)
{
    return with_kernel(group, zero, [&](auto kernel, int threads, int smem) {
        return launch_grid(kernel, p, grid, threads, smem, stream, cooperative, pdl);
    });
}

}  // namespace tovl
