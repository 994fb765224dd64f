// moe_decode.cu -- a whole gated expert layer for up to 64 tokens in one kernel
// (moe_direct.cu has the small ones; use_direct_moe is the rule).
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
// What bounds it: the weights' stream (13 tokens, 4 of 32 experts of 7168 x 2048,
// bf16, 2.3 GB: 356 us, 6.5 TB/s; 64 tokens, 2.8 GB: 452 us; 4-bit, 24 tokens, 2 of 8
// of 4096 x 2048, 110 MB: 45.9 us, instructions) and about 14 us that do not depend
// on it: launch and tables 4.5, three barriers 1 each, the sums of the parts 2 and
// 1.5, the CTAs' different ends 2 to 6 (4-bit, 1 token, 4 experts of 7168 x 2048, 91
// MB: 33.0 us).
//
// Roundings: x and the weights are bf16 (or 4-bit with their scales applied
// in fp32), sums are fp32.  With bf16 weights h is split into two bf16
// numbers, its rounding and the rest, and the second product multiplies both
// (the second one rides on the same weight fragments): one bf16 h would raise
// the error of the result from its own rounding's 1.7e-3 to 2.4e-3, the pair
// leaves it alone.  With 4-bit weights h is fp16 with a power of two per 128
// columns, 11 significant bits: 2^-11 of a number at most.  The roundings of a
// sum's I numbers are independent, about 1.1e-4 of the result together, beside the
// 1.66e-3 of its own rounding (measured with it: 1.67e-3); a second part would
// double the products, which bound the 4-bit form.
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
    int n_entries, n_rows, bad;
};

// What only building the tables needs; lies where the rows go later.
struct Building {
    unsigned long long mask[kMaxExperts];   // tokens of each expert
    float gate[kMaxPairs];
    int16_t topk[kMaxPairs];
};
static_assert(sizeof(Building) <= kRowBuffers, "the tables' scratch fits the row buffers");

// Rows of an expert that one entry takes: 4-bit blocks keep the sums of a
// scale group beside the running ones.
constexpr int pass_rows(int group) { return group ? 16 : 64; }

template <int G>
constexpr int smem_size() { return 1024 + Shape<G>::kRing + kRowBuffers + static_cast<int>(sizeof(Tables)) + 16; }

// Builds the list of experts with rows.  Every CTA builds the same list
// (ascending experts, ascending tokens), so they agree on row numbers without
// talking.  A token that names an expert twice has one row with both weights.
// False if an id is outside [-1, E).
template <int PASS, int THREADS>
__device__ bool build_tables(const MoeParams& p, Tables& tb, Building& bd)
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
    for (int e = tid; e < p.E; e += THREADS) bd.mask[e] = 0;
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
            bd.topk[i] = static_cast<int16_t>(id[u]);
            bd.gate[i] = w[u];
            if (id[u] >= 0) atomicOr(bd.mask + id[u], 1ull << (i / p.k));
        }
    }
    __syncthreads();
    if (tb.bad) return false;
    if (tid < 32) {
        int n = 0, rows = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            unsigned long long m = e < p.E ? bd.mask[e] : 0;
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
__device__ void build_pairs(const MoeParams& p, Tables& tb, const Building& bd)
{
    for (int i = threadIdx.x; i < p.T * p.k; i += THREADS) tb.pair_row[i] = -1;
    __syncthreads();
    for (int r = threadIdx.x; r < tb.n_rows; r += THREADS) {
        const int e = entry_expert(tb.entry[tb.row_entry[r]]), t = tb.row_tok[r];
        int first = -1;
        float w = 0.f;
        for (int j = 0; j < p.k; ++j)
            if (bd.topk[t * p.k + j] == e) {
                if (first < 0) first = j;
                w += bd.gate[t * p.k + j];
            }
        tb.pair_row[t * p.k + first] = static_cast<int16_t>(r);
        tb.pair_w[t * p.k + first] = w;
    }
}

struct Calls {
    const MoeParams& p;
    const Tables& tb;
    __device__ __forceinline__ const WeightMaps* maps(int ph) const { return ph ? &p.w2 : &p.w13; }
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
        constexpr Rows kind = !H ? Rows::kBf16 : G ? Rows::kHalf : Rows::kPair;
        eng.template segment<NT, kind>(
            i0, i1, part, N, cnt, tile * kTileCols, N, K,
            [&](int r, int k, bool lo) {
                if (H) {     // (written in this launch)
                    const uint16_t* h = static_cast<const uint16_t*>(lo ? p.h_lo : p.h_hi);
                    return __ldcg(reinterpret_cast<const uint4*>(h + static_cast<long long>(off + r) * p.I + k));
                }
                return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + tb.row_tok[off + r] * p.ldx + k));
            },
            [&](int r, int k) { return __ldcg(static_cast<const float*>(p.h_lo) + (off + r) * scale_groups() + k / kXScaleGroup); });
    }

    // 4-bit weights: h_lo holds the scales of h, fp32 [row][ceil(I / 128)]
    __device__ __forceinline__ int scale_groups() const { return (p.I + kXScaleGroup - 1) / kXScaleGroup; }

    template <bool H>
    __device__ __forceinline__ void product()
    {
        eng.walk(H, [&](int matrix, int tile, int i0, int i1, int number) {
            const uint32_t en = tb.entry[matrix];
            const int cnt = entry_rows(en);
            if (cnt <= 8) segment<1, H>(en, tile, i0, i1, number);
            else if (cnt <= 16) segment<2, H>(en, tile, i0, i1, number);
            else if constexpr (G == 0) {
                if (cnt <= 32) segment<4, H>(en, tile, i0, i1, number);
                else segment<8, H>(en, tile, i0, i1, number);
            }
        });
    }

    // Where the parts of column n of a row of product `ph` start, and their number.
    __device__ __forceinline__ const float* parts(int ph, int row, int n, int N, int& count) const
    {
        const Product& q = tb.pr[ph];
        count = q.parts((tb.row_entry[row] * q.tiles + n / kTileCols) * q.kb);
        return p.part + static_cast<long long>(row) * N + n;
    }

    // A warp takes 128 columns of a row at a time, a lane four.
    __device__ __forceinline__ void activations()
    {
        const int groups = scale_groups();
        const long long stride = static_cast<long long>(p.T) * p.k * 2 * p.I;
        const int lane = threadIdx.x & 31;
        for (int i = spread_thread() >> 5; i < tb.n_rows * groups; i += gridDim.x * P::kWarps) {
            const int row = i / groups, n = (i - row * groups) * kXScaleGroup + lane * 4;
            const bool in = n < p.I;
            int count[2];
            const float* part[2] = {parts(0, row, in ? n : 0, 2 * p.I, count[0]), parts(0, row, p.I + (in ? n : 0), 2 * p.I, count[1])};
            float4 s[2];
            add_parts<2>(s, part, count, stride);
            const float g[4] = {s[0].x, s[0].y, s[0].z, s[0].w}, u[4] = {s[1].x, s[1].y, s[1].z, s[1].w};
            float h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = in ? g[j] / (1.f + expf(-g[j])) * u[j] : 0.f;
            const long long at = static_cast<long long>(row) * p.I + n;
            if constexpr (G != 0) {
                uint32_t e = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) e = max(e, (__float_as_uint(h[j]) >> 23) & 255u);
                e = __reduce_max_sync(0xffffffffu, e);
                const float f = half_scale(e);
                if (in)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.h_hi) + at) =
                        make_uint2(pack_h2(h[0] * f, h[1] * f), pack_h2(h[2] * f, h[3] * f));
                if (lane == 0) static_cast<float*>(p.h_lo)[i] = half_unscale(e);
            } else if (in) {
                float hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    hi[j] = __bfloat162float(__float2bfloat16(h[j]));
                    // (an overflowed h has no second part)
                    lo[j] = fabsf(h[j] - hi[j]) < INFINITY ? h[j] - hi[j] : 0.f;
                }
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.h_hi) + at) =
                    make_uint2(ptx::pack_bf16x2(hi[0], hi[1]), ptx::pack_bf16x2(hi[2], hi[3]));
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.h_lo) + at) =
                    make_uint2(ptx::pack_bf16x2(lo[0], lo[1]), ptx::pack_bf16x2(lo[2], lo[3]));
            }
        }
    }

    // Four columns of a token to a thread; with few tokens to up to eight
    // neighbouring lanes, which share out its experts (one token, four experts
    // of 7168 columns: 3.0 us with one lane, 1.5 with four).
    __device__ __forceinline__ void outputs()
    {
        const int quads = p.H / 4, total = p.T * quads;
        const long long stride = static_cast<long long>(p.T) * p.k * p.H;
        const int threads = gridDim.x * P::kThreads, me = spread_thread();
        int log = 0;
        while (log < 3 && 1 << log < p.k && total << (log + 1) <= threads) ++log;
        const int lanes = 1 << log, own = me & (lanes - 1);
        for (int base = (me & ~31) >> log; base < total; base += threads >> log) {       // (a warp goes on together)
            const int i = base + ((me & 31) >> log), q = min(i, total - 1), t = q / quads, n = (q - t * quads) * 4;
            float4 out4 = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j = own; j < p.k; j += 2 * lanes) {      // two slots' parts together
                const float* part[2];
                int count[2];
                float w[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int slot = j + u * lanes, row = slot < p.k ? tb.pair_row[t * p.k + slot] : -1;
                    part[u] = p.part;
                    count[u] = 0;
                    w[u] = 0.f;
                    if (row >= 0) {
                        part[u] = parts(1, row, n, p.H, count[u]);
                        w[u] = tb.pair_w[t * p.k + slot];
                    }
                }
                float4 s[2];
                add_parts<2>(s, part, count, stride);
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (count[u])
                        out4.x += w[u] * s[u].x, out4.y += w[u] * s[u].y, out4.z += w[u] * s[u].z, out4.w += w[u] * s[u].w;
            }
            for (int d = 1; d < lanes; d *= 2) {
                out4.x += __shfl_xor_sync(0xffffffffu, out4.x, d), out4.y += __shfl_xor_sync(0xffffffffu, out4.y, d);
                out4.z += __shfl_xor_sync(0xffffffffu, out4.z, d), out4.w += __shfl_xor_sync(0xffffffffu, out4.w, d);
            }
            if (own > 0 || i >= total) continue;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + t * p.ldo + n;
            if (p.out_vec) {
                *reinterpret_cast<uint2*>(out) = make_uint2(ptx::pack_bf16x2(out4.x, out4.y), ptx::pack_bf16x2(out4.z, out4.w));
            } else {
                out[0] = __float2bfloat16(out4.x), out[1] = __float2bfloat16(out4.y);
                out[2] = __float2bfloat16(out4.z), out[3] = __float2bfloat16(out4.w);
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
    Building& bd = *reinterpret_cast<Building*>(rows_buf);
    const Calls calls{p, tb};
    Engine<G, Z, Calls> eng{calls, tb.pr, tb.queue, p.sync + kTicketWord, p.ctrl, p.pipe_timeout_ns, 2};
    eng.warp = threadIdx.x >> 5;
    eng.lane = threadIdx.x & 31;
    eng.init(smem, rows_buf);
    if (threadIdx.x == 0) {
        ptx::prefetch_tmap(&p.w13.w);
        ptx::prefetch_tmap(&p.w2.w);
    }
    for (int i = threadIdx.x; i < 2 * (kMaxItems + 8); i += P::kThreads)
        tb.queue[i / (kMaxItems + 8)].item[i % (kMaxItems + 8)] = kNoItem;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int grid = gridDim.x;
    if (!build_tables<pass_rows(G), P::kThreads>(p, tb, bd)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_error(p.ctrl, kErrInvalid);
        return;
    }
    if (threadIdx.x < 2)
        tb.pr[threadIdx.x].init(tb.n_entries, threadIdx.x ? p.H : 2 * p.I, threadIdx.x ? p.I : p.H, P::kRows, P::kUnitBytes, grid,
                               p.most_parts);
    __syncthreads();
    eng.start();
    build_pairs<P::kThreads>(p, tb, bd);
    __syncthreads();       // (the scratch becomes row buffers)
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
        for (int i = 0; i <= kExitWord; i += kSyncStep) ptx::st_relaxed_gpu(p.sync + i, 0);
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
