// moe_decode.cu -- a whole gated expert layer for up to 64 tokens in one kernel.
//
//   h[t, e]  = silu(x[t] W13[e][:, :I]) * (x[t] W13[e][:, I:])      for the experts e that token t names
//   out[t]   = sum over those e of gate[t, e] * (h[t, e] W2[e])
//
// One persistent grid, one CTA per SM.  Phase 1 streams the W13 blocks of the
// experts that some token names, phase 2 their W2 blocks, each split evenly
// over the CTAs (skinny.cuh); the rings of weight stages run straight through
// from one phase into the next, so the memory system keeps delivering W2 while
// the CTAs meet at the one barrier between the phases (a count of finished
// phase-1 tiles that every CTA waits for).
//
// Block order.  Phase 1: (expert, tile of 64 gate columns and the 64 up
// columns that go with them, k, gate | up): even warps sum gate, odd warps up,
// and a whole tile's activations are formed where its sums meet.  Phase 2:
// (tile of 64 output columns, expert, k): a CTA adds the experts of a column
// tile in shared memory, in ascending order, weighted in fp32.
//
// Roundings: x and the weights are bf16 (or 4-bit with their scales applied
// in fp32), sums are fp32.  h is split into two bf16 numbers, its rounding
// and the rest, and phase 2 multiplies both (the second product rides on the
// same weight fragments): one bf16 h would double the error of the result's
// own rounding (1.7e-3 -> 2.4e-3 relative), the pair leaves it alone.
#include "launch.cuh"
#include "skinny.cuh"

namespace tovl {

namespace {

using namespace skinny;
constexpr int kCta = skinny::kThreads;

// Rows that one pass over an expert's weights takes.  4-bit blocks keep the
// sums of a scale group beside the running ones and both halves of the
// activations of 128 rows of W in registers, which leaves room for 16 rows;
// an expert with more rows is listed once per 16.
template <bool Q4>
constexpr int kPassRows = Q4 ? 16 : 64;

constexpr int kMaxPairs = kMaxDecodeRows * kMaxDecodeK;
constexpr int kMaxEntries = kMaxExperts + kMaxPairs / 16;

// An expert (or 16 rows of one) that phase 1 and 2 go through.
__device__ __forceinline__ uint32_t pack_entry(int e, int cnt, int off) { return e | (cnt - 1) << 10 | off << 16; }
__device__ __forceinline__ int entry_expert(uint32_t v) { return v & 1023; }
__device__ __forceinline__ int entry_rows(uint32_t v) { return ((v >> 10) & 63) + 1; }
__device__ __forceinline__ int entry_off(uint32_t v) { return v >> 16; }

struct Tables {
    float acc[kMaxDecodeRows * kCols];      // phase 2: output tile of this CTA's experts so far
    float row_w[kMaxPairs];                 // gate weight of each (expert, token) row
    uint32_t entry[kMaxEntries];
    uint8_t row_tok[kMaxPairs];
    uint64_t mask[kMaxExperts];             // tokens of each expert
    int n_entries, bad, flag;
};

template <bool Q4>
constexpr int smem_size() { return base_smem(Q4) + static_cast<int>(sizeof(Tables)); }

// Position in a block list: `top` slowest, then `mid`, then `i`.
struct Cursor {
    int left;            // blocks of this warp still to come
    int i, mid, top, ni, nmid;
    __device__ void init(int start, int end, int ni_, int nmid_)
    {
        ni = ni_;
        nmid = nmid_;
        left = end > start ? (end - start + kWarps - 1) / kWarps : 0;
        i = start % ni;
        const int r = start / ni;
        mid = r % nmid;
        top = r / nmid;
    }
    __device__ void next()
    {
        --left;
        i += kWarps;
        while (i >= ni) {
            i -= ni;
            if (++mid == nmid) {
                mid = 0;
                ++top;
            }
        }
    }
};

// Builds the list of experts with rows, each row's token and weight.  Every
// CTA builds the same list (ascending experts, ascending tokens), so they
// agree on row numbers without talking.  A token that names an expert twice
// has one row with both weights.  False if an id is outside [-1, E).
template <bool Q4>
__device__ bool build_tables(const MoeParams& p, Tables& tb)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const int pairs = p.T * p.k;
    for (int e = tid; e < p.E; e += kCta) tb.mask[e] = 0;
    if (tid == 0) tb.bad = 0;
    __syncthreads();
    int mine[kMaxPairs / kCta];
#pragma unroll
    for (int u = 0; u < kMaxPairs / kCta; ++u) {
        const int i = tid + u * kCta;
        mine[u] = i < pairs ? __ldg(p.topk + i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kMaxPairs / kCta; ++u) {
        const int i = tid + u * kCta;
        if (mine[u] < -1 || mine[u] >= p.E) {
            tb.bad = 1;
            mine[u] = -1;
        }
        if (mine[u] >= 0) atomicOr(reinterpret_cast<unsigned long long*>(tb.mask + mine[u]), 1ull << (i / p.k));
    }
    __syncthreads();
    if (tb.bad) return false;
    if (tid < 32) {
        int n = 0, rows = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            const int cnt = e < p.E ? __popcll(tb.mask[e]) : 0;
            const int passes = (cnt + kPassRows<Q4> - 1) / kPassRows<Q4>;
            int sn = passes, sr = cnt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, sn, d), b = __shfl_up_sync(0xffffffffu, sr, d);
                if (lane >= d) {
                    sn += a;
                    sr += b;
                }
            }
            int at = n + sn - passes, off = rows + sr - cnt;
            for (int q = cnt; q > 0; q -= kPassRows<Q4>, ++at, off += kPassRows<Q4>)
                tb.entry[at] = pack_entry(e, q < kPassRows<Q4> ? q : kPassRows<Q4>, off);
            // row numbers start where the expert's first entry does
            off = rows + sr - cnt;
            uint64_t m = cnt ? tb.mask[e] : 0;
            for (int r = 0; m; ++r, m &= m - 1) tb.row_tok[off + r] = static_cast<uint8_t>(__ffsll(m) - 1);
            n += __shfl_sync(0xffffffffu, sn, 31);
            rows += __shfl_sync(0xffffffffu, sr, 31);
        }
        if (lane == 0) tb.n_entries = n;
    }
    __syncthreads();
    return true;
}

// The gate weight of every row: the sum over the token's slots that name the
// row's expert, in ascending slots.
__device__ void build_weights(const MoeParams& p, Tables& tb)
{
    for (int a = threadIdx.x >> 5; a < tb.n_entries; a += kWarps) {
        const uint32_t en = tb.entry[a];
        const int e = entry_expert(en), off = entry_off(en), cnt = entry_rows(en);
        for (int r = threadIdx.x & 31; r < cnt; r += 32) {
            const int t = tb.row_tok[off + r];
            float w = 0.f;
            for (int j = 0; j < p.k; ++j)
                if (__ldg(p.topk + t * p.k + j) == e) w += __ldg(p.gate_w + t * p.k + j);
            tb.row_w[off + r] = w;
        }
    }
}

template <bool Q4>
struct Worker {
    const MoeParams& p;
    Tables& tb;
    float* red;
    Ring<Q4> ring;
    Cursor f1, f2;       // blocks to fetch, per phase
    int warp, lane;
    uint64_t pol;

    static constexpr int KR = block_rows(Q4);

    // lane 0: fetch the warp's next block, of either phase
    __device__ __forceinline__ void fetch()
    {
        if (f1.left > 0) {
            if (lane == 0) {
                const uint32_t en = tb.entry[f1.top];
                ring.issue(p.w13, ((f1.i & 1) ? p.I : 0) + f1.mid * kCols, (f1.i >> 1) * KR, entry_expert(en), p.group,
                           p.has_zero, pol);
            }
            ring.filled();
            f1.next();
        } else if (f2.left > 0) {
            if (lane == 0)
                ring.issue(p.w2, f2.top * kCols, f2.i * KR, entry_expert(tb.entry[f2.mid]), p.group, p.has_zero, pol);
            ring.filled();
            f2.next();
        }
    }

    // Sums of the warp's share of blocks [i0, i1) of a tile: first is the
    // warp's first block in it.  PH2: rows come from h (two parts).
    template <int NT, bool PH2>
    __device__ __forceinline__ void blocks(float (&acc)[4][NT][4], int first, int i1, uint32_t en)
    {
        const int g = lane >> 2, t = lane & 3;
        const int cnt = entry_rows(en), off = entry_off(en);
        const int K = PH2 ? p.I : p.H;
        const __nv_bfloat16* row[NT];
        const long long lo = static_cast<const __nv_bfloat16*>(p.h_lo) - static_cast<const __nv_bfloat16*>(p.h_hi);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // a row past the last one repeats row 0; its column is never stored
            const int r = nt * 8 + g < cnt ? nt * 8 + g : 0;
            if (PH2) row[nt] = static_cast<const __nv_bfloat16*>(p.h_hi) + static_cast<long long>(off + r) * p.I;
            else row[nt] = static_cast<const __nv_bfloat16*>(p.x) + tb.row_tok[off + r] * p.ldx;
        }
        const uint4 none = make_uint4(0, 0, 0, 0);
        for (int i = first; i < i1; i += kWarps) {
            const int k0 = (PH2 ? i : i >> 1) * KR + 8 * t;
            if constexpr (Q4) {
                uint4 b[4][NT], bl[4][NT];
                float2 sx[NT];
#pragma unroll
                for (int R = 0; R < 4; ++R)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int k = k0 + 32 * R;
                        const bool in = k < K;
                        if (PH2) {
                            b[R][nt] = in ? __ldcg(reinterpret_cast<const uint4*>(row[nt] + k)) : none;
                            bl[R][nt] = in ? __ldcg(reinterpret_cast<const uint4*>(row[nt] + lo + k)) : none;
                        } else {
                            b[R][nt] = in ? __ldg(reinterpret_cast<const uint4*>(row[nt] + k)) : none;
                        }
                    }
                ring.wait(p.ctrl, p.pipe_timeout_ns);
                block_q4<NT, PH2, false>(acc, b, bl, sx, ring.stage(), ring.stage_meta(), p.group / 32, p.has_zero, lane);
            } else {
                uint4 b[NT], bl[NT];
                const bool in = k0 < K;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (PH2) {
                        b[nt] = in ? __ldcg(reinterpret_cast<const uint4*>(row[nt] + k0)) : none;
                        bl[nt] = in ? __ldcg(reinterpret_cast<const uint4*>(row[nt] + lo + k0)) : none;
                    } else {
                        b[nt] = in ? __ldg(reinterpret_cast<const uint4*>(row[nt] + k0)) : none;
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    b[nt] = rotate_pairs(b[nt], t);
                    if (PH2) bl[nt] = rotate_pairs(bl[nt], t);
                }
                ring.wait(p.ctrl, p.pipe_timeout_ns);
                block_bf16<NT, PH2>(acc, b, bl, ring.stage(), lane);
            }
            ring.taken();
            __syncwarp();      // every lane has read the stage before it is filled again
            fetch();
        }
    }

    // h of one row and column, in two bf16 parts
    __device__ __forceinline__ void store_h(int row, int col, float gate, float up)
    {
        const float h = gate / (1.f + expf(-gate)) * up;
        const __nv_bfloat16 hi = __float2bfloat16(h);
        const long long at = static_cast<long long>(row) * p.I + col;
        static_cast<__nv_bfloat16*>(p.h_hi)[at] = hi;
        // (an overflowed h has no second part)
        const float rest = h - __bfloat162float(hi);
        static_cast<__nv_bfloat16*>(p.h_lo)[at] = __float2bfloat16(fabsf(rest) < INFINITY ? rest : 0.f);
    }

    // One tile of phase 1, or the part of it that this CTA owns: `part` is
    // null for a whole tile, else where [64 rows][gate 64 | up 64] goes.
    template <int NT>
    __device__ __forceinline__ void tile1(int first, int i1, uint32_t en, int c, float* part)
    {
        float acc[4][NT][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
        blocks<NT, false>(acc, first, i1, en);
        const int cnt = entry_rows(en), off = entry_off(en);
        const int col = threadIdx.x & 63, q = threadIdx.x >> 6;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt * 8 >= cnt) break;
            store_red<Q4, NT>(red, acc, nt, warp, lane);
            __syncthreads();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = q + 4 * u, row = nt * 8 + r;
                float gate = 0.f, up = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; w += 2) {
                    gate += red[(w * 8 + r) * kRedPitch + col];
                    up += red[((w + 1) * 8 + r) * kRedPitch + col];
                }
                if (row < cnt) {
                    if (part) {
                        part[row * (2 * kCols) + col] = gate;
                        part[row * (2 * kCols) + kCols + col] = up;
                    } else if (c * kCols + col < p.I) {
                        store_h(off + row, c * kCols + col, gate, up);
                    }
                }
            }
            __syncthreads();
        }
    }

    // The experts' part of an output tile: acc[token][column] += weight * row
    template <int NT>
    __device__ __forceinline__ void tile2(int first, int i1, uint32_t en)
    {
        float acc[4][NT][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
        blocks<NT, true>(acc, first, i1, en);
        const int cnt = entry_rows(en), off = entry_off(en);
        const int col = threadIdx.x & 63, q = threadIdx.x >> 6;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt * 8 >= cnt) break;
            store_red<Q4, NT>(red, acc, nt, warp, lane);
            __syncthreads();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = q + 4 * u, row = nt * 8 + r;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += red[(w * 8 + r) * kRedPitch + col];
                // the rows of an expert are different tokens
                if (row < cnt) tb.acc[tb.row_tok[off + row] * kCols + col] += tb.row_w[off + row] * v;
            }
            __syncthreads();
        }
    }
};

// Smallest n-tile count of a pass.
template <bool Q4, class F1, class F2, class F4, class F8>
__device__ __forceinline__ void by_rows(int cnt, F1 f1, F2 f2, F4 f4, F8 f8)
{
    if (cnt <= 8) f1();
    else if (cnt <= 16) f2();
    else if constexpr (!Q4) {
        if (cnt <= 32) f4();
        else f8();
    }
}

template <bool Q4>
__global__ void __launch_bounds__(kCta, 1) moe_decode_kernel(const __grid_constant__ MoeParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    float* red = reinterpret_cast<float*>(smem + ring_bytes(Q4) + meta_bytes(Q4));
    Tables& tb = *reinterpret_cast<Tables*>(smem + base_smem(Q4) - 1024);
    Worker<Q4> w{p, tb, red};
    w.warp = threadIdx.x >> 5;
    w.lane = threadIdx.x & 31;
    w.pol = ptx::l2_policy(0);
    w.ring.init(smem, w.warp);
    if (w.lane == 0) {
        w.ring.init_barriers();
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.w13.w);
        ptx::prefetch_tmap(&p.w2.w);
    }
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int grid = gridDim.x, cta = blockIdx.x;
    if (!build_tables<Q4>(p, tb)) {
        if (cta == 0 && threadIdx.x == 0) record_error(p.ctrl, kErrInvalid);
        return;
    }
    const int nA = tb.n_entries;
    constexpr int KR = block_rows(Q4);
    const int tiles1 = (p.I + kCols - 1) / kCols, tiles2 = (p.H + kCols - 1) / kCols;
    const int len1 = 2 * ((p.H + KR - 1) / KR);           // blocks of a phase-1 tile
    const int kb2 = (p.I + KR - 1) / KR, len2 = nA * kb2; // blocks of an expert's part and of a phase-2 tile
    const int total1 = nA * tiles1 * len1, total2 = tiles2 * len2;
    const int per1 = blocks_per_cta(total1, grid), per2 = blocks_per_cta(total2, grid);
    const int b1 = min(cta * per1, total1), e1 = min(b1 + per1, total1);
    const int b2 = min(cta * per2, total2), e2 = min(b2 + per2, total2);
    w.f1.init(b1 + w.warp, e1, len1, tiles1);
    w.f2.init(b2 + w.warp, e2, nA ? kb2 : 1, nA ? nA : 1);
#pragma unroll 1
    for (int s = 0; s < Ring<Q4>::S; ++s) w.fetch();
    build_weights(p, tb);

    // ---------------------------------------------------------------- phase 1
    int done = 0;
    for (int b = b1; b < e1;) {
        const int tile = b / len1, t0 = tile * len1, t1 = t0 + len1;
        const int end = min(t1, e1);
        const uint32_t en = tb.entry[tile / tiles1];
        const int c = tile % tiles1;
        const bool whole = b == t0 && end == t1;
        float* part = whole ? nullptr
                            : p.part1 + (static_cast<long long>(cta) * 2 + (b == b1 ? 0 : 1)) * (kMaxDecodeRows * 2 * kCols);
        // the warp's first block here, as an index inside the tile
        const int first = b - t0 + ((w.warp - (b - b1)) & (kWarps - 1));
        by_rows<Q4>(
            entry_rows(en), [&] { w.template tile1<1>(first, end - t0, en, c, part); },
            [&] { w.template tile1<2>(first, end - t0, en, c, part); },
            [&] { w.template tile1<4>(first, end - t0, en, c, part); },
            [&] { w.template tile1<8>(first, end - t0, en, c, part); });
        if (whole) {
            ++done;
        } else {
            const int c0 = t0 / per1, c1 = (t1 - 1) / per1;
            if (last_arrival(p.sync + c0, c1 - c0 + 1, &tb.flag)) {
                const int cnt = entry_rows(en), off = entry_off(en);
                const int col = threadIdx.x & 63;
                if (c * kCols + col < p.I) {
                    for (int r = threadIdx.x >> 6; r < cnt; r += kCta / kCols) {
                        float gate = 0.f, up = 0.f;
                        for (int k = c0; k <= c1; ++k) {
                            const float* s = p.part1 +
                                             (static_cast<long long>(k) * 2 + (t0 <= k * per1 ? 0 : 1)) * (kMaxDecodeRows * 2 * kCols) +
                                             r * (2 * kCols) + col;
                            gate += __ldcg(s);
                            up += __ldcg(s + kCols);
                        }
                        w.store_h(off + r, c * kCols + col, gate, up);
                    }
                }
                ++done;
            }
        }
        b = end;
    }
    // every CTA announces its finished tiles, then waits for all of them
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (done) ptx::red_add_release_gpu(p.sync + kReadyWord, done);
        const int target = nA * tiles1 + p.ready_offset;
        const uint64_t start = ptx::globaltimer();
        for (int spin = 1; ptx::ld_acquire_gpu(p.sync + kReadyWord) < target; ++spin) {
            if ((spin & 63) == 0 && ptx::globaltimer() - start > static_cast<uint64_t>(p.timeout_ns)) {
                record_error(p.ctrl, kErrTimeout);
                break;
            }
        }
        // the last CTA to leave clears both counts for the next call
        if (ptx::atom_add_relaxed_gpu(p.sync + kExitWord, 1) == grid - 1) {
            ptx::st_relaxed_gpu(p.sync + kReadyWord, 0);
            ptx::st_relaxed_gpu(p.sync + kExitWord, 0);
        }
        __threadfence();
    }
    __syncthreads();

    // ---------------------------------------------------------------- phase 2
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    const int col = threadIdx.x & 63, q = threadIdx.x >> 6;
    if (nA == 0) {       // no token names an expert
        for (int c = cta; c < tiles2; c += grid)
            if (c * kCols + col < p.H)
                for (int t = q; t < p.T; t += kCta / kCols) out[t * p.ldo + c * kCols + col] = __float2bfloat16(0.f);
        return;
    }
    for (int b = b2; b < e2;) {
        const int c = b / len2, t0 = c * len2, t1 = t0 + len2;
        const int end = min(t1, e2);
        for (int i = threadIdx.x; i < p.T * kCols; i += kCta) tb.acc[i] = 0.f;
        __syncthreads();
        for (int s = b; s < end;) {
            const int a = (s - t0) / kb2, s0 = t0 + a * kb2;
            const int se = min(s0 + kb2, end);
            const uint32_t en = tb.entry[a];
            const int first = s - s0 + ((w.warp - (s - b2)) & (kWarps - 1));
            by_rows<Q4>(
                entry_rows(en), [&] { w.template tile2<1>(first, se - s0, en); },
                [&] { w.template tile2<2>(first, se - s0, en); }, [&] { w.template tile2<4>(first, se - s0, en); },
                [&] { w.template tile2<8>(first, se - s0, en); });
            s = se;
        }
        const bool in = c * kCols + col < p.H;
        if (b == t0 && end == t1) {
            if (in)
                for (int t = q; t < p.T; t += kCta / kCols)
                    out[t * p.ldo + c * kCols + col] = __float2bfloat16(tb.acc[t * kCols + col]);
        } else {
            const long long stride = static_cast<long long>(p.T) * kCols;
            float* part = p.part2 + (static_cast<long long>(cta) * 2 + (b == b2 ? 0 : 1)) * stride;
            for (int i = threadIdx.x; i < p.T * kCols; i += kCta) part[i] = tb.acc[i];
            const int c0 = t0 / per2, c1 = (t1 - 1) / per2;
            if (last_arrival(p.sync + kMaxGrid + c0, c1 - c0 + 1, &tb.flag) && in) {
                for (int t = q; t < p.T; t += kCta / kCols) {
                    float v = 0.f;
                    for (int k = c0; k <= c1; ++k)
                        v += __ldcg(p.part2 + (static_cast<long long>(k) * 2 + (t0 <= k * per2 ? 0 : 1)) * stride + t * kCols + col);
                    out[t * p.ldo + c * kCols + col] = __float2bfloat16(v);
                }
            }
        }
        __syncthreads();
        b = end;
    }
}

}  // namespace

cudaError_t prepare_moe_decode()
{
    cudaError_t e = cudaFuncSetAttribute(moe_decode_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_size<false>());
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(moe_decode_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_size<true>());
    return e;
}

cudaError_t launch_moe_decode(const MoeParams& p, bool q4, int grid, cudaStream_t stream, bool cooperative, bool pdl)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(kCta);
    lc.dynamicSmemBytes = q4 ? smem_size<true>() : smem_size<false>();
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = cooperative ? 1 : 0;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = pdl ? 2 : 1;
    return q4 ? cudaLaunchKernelEx(&lc, moe_decode_kernel<true>, p) : cudaLaunchKernelEx(&lc, moe_decode_kernel<false>, p);
}

}  // namespace tovl
