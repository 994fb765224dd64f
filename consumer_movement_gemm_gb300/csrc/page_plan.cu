// page_plan.cu -- pages, cache slots and positions of a step's new tokens.
//
// Every CTA scans all requests' counts for itself (prefix sums of new tokens,
// of pages taken and of pages given back, in shared memory) and works on a
// share of the outputs: a token or a page finds its request by bisection.
// Pages are taken from the ring's head in the order of the requests, so a
// token's page is known from the sums alone and nothing waits for the table.
// Given-back pages go behind the ring's tail, which no taken page lies at.
// A thread looks for a token, a taken page and a given-back page at once, so
// that their dependent loads overlap.  What is updated in place (lengths,
// state) is written by the CTA that finishes last, when all others have read it.
//
// What bounds it: latency (a launch, the loads of the counts, the sums, the
// bisections, the loads of ring and table): 256 requests with one token each 3.5
// us, prompts of 62000 tokens 4.1 us.
#include "common.cuh"
#include "paged.cuh"
#include "sync.cuh"

namespace tovl {

namespace {

constexpr unsigned kMostSum = 0x7fffffffu;       // the sums stop there

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlanParams p)
{
    constexpr int kPlanWarps = kPlanThreads / 32;
    extern __shared__ int sums[];          // lengths; inclusive sums: tokens, pages taken, pages given back
    __shared__ unsigned s_warp[3][kPlanWarps];
    __shared__ int s_last;
    int* const held = sums;
    int* const tok_end = sums + p.B;
    int* const take_end = sums + 2 * p.B;
    int* const back_end = sums + 3 * p.B;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned page = p.page;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    const auto over_page = [&](unsigned tokens) { return p.page_shift >= 0 ? tokens >> p.page_shift : tokens / page; };
    const auto pages_for = [&](unsigned tokens) { return over_page(tokens + page - 1); };
    const int per = (p.B + kPlanThreads - 1) / kPlanThreads, b0 = tid * per, b1 = min(p.B, b0 + per);
    const int head = __ldcg(p.state), free = __ldcg(p.state + 1);
    const long long most = min(static_cast<long long>(p.width) * p.page, 0x7fffffffLL);
    unsigned sum[3] = {0, 0, 0};
    bool bad = head < 0 || head >= p.pages || free < 0 || free > p.pages;
    for (int b = b0; b < b1; ++b) {
        const int len = __ldcg(p.length + b), add = __ldcg(p.add + b);
        held[b] = len, tok_end[b] = add;
        if (len < 0 || add < -1 || static_cast<long long>(len) + max(add, 0) > most) {
            bad = true;
            continue;
        }
        const unsigned have = pages_for(len);
        sum[0] = min(sum[0] + max(add, 0), kMostSum);
        sum[1] = min(sum[1] + (add > 0 ? pages_for(len + add) - have : 0), kMostSum);
        sum[2] = min(sum[2] + (add < 0 ? have : 0), kMostSum);
    }
    unsigned before[3], total[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) before[k] = sum[k];
#pragma unroll
    for (int d = 1; d < 32; d *= 2)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const unsigned o = __shfl_up_sync(0xffffffffu, before[k], d);
            if (lane >= d) before[k] = min(before[k] + o, kMostSum);
        }
    if (lane == 31) s_warp[0][warp] = before[0], s_warp[1][warp] = before[1], s_warp[2][warp] = before[2];
    bad = __syncthreads_or(bad);
    // (the sums of the warps, a lane each)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        unsigned w = lane < kPlanWarps ? s_warp[k][lane] : 0;
#pragma unroll
        for (int d = 1; d < kPlanWarps; d *= 2) {
            const unsigned o = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w = min(w + o, kMostSum);
        }
        total[k] = __shfl_sync(0xffffffffu, w, kPlanWarps - 1);
        const unsigned base = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
        before[k] = before[k] - sum[k] + (warp ? base : 0);        // (right where no sum has stopped: other calls do nothing)
    }
    bad = bad || total[0] > static_cast<unsigned>(p.cap) || total[2] == kMostSum || static_cast<unsigned>(free) + total[2] > static_cast<unsigned>(p.pages);
    const int lacking = bad ? -1 : total[1] > static_cast<unsigned>(free) ? static_cast<int>(total[1] - free) : 0;
    const bool go = lacking == 0;
    if (go) {
        unsigned run[3] = {before[0], before[1], before[2]};
        for (int b = b0; b < b1; ++b) {
            const int len = held[b], add = tok_end[b];
            const unsigned have = pages_for(len);
            run[0] += max(add, 0);
            run[1] += add > 0 ? pages_for(len + add) - have : 0;
            run[2] += add < 0 ? have : 0;
            tok_end[b] = run[0], take_end[b] = run[1], back_end[b] = run[2];
            if (!p.in_place && blockIdx.x == 0) p.length_out[b] = add < 0 ? 0 : len + add;
        }
    } else {
        if (bad && blockIdx.x == 0 && tid == 0) record_error(p.ctrl, kErrInvalid);
        if (!p.in_place && blockIdx.x == 0)
            for (int b = b0; b < b1; ++b) p.length_out[b] = held[b];
    }
    __syncthreads();

    const int tokens = go ? total[0] : 0, takes = go ? total[1] : 0, backs = go ? total[2] : 0;
    const auto in_ring = [&](unsigned i) { return i >= static_cast<unsigned>(p.pages) ? i - p.pages : i; };
    const unsigned tail = in_ring(static_cast<unsigned>(head) + free);
    const long long items = max(max(max(p.cap, takes), backs), p.B + 1), step = static_cast<long long>(gridDim.x) * kPlanThreads;
    int top = 1;
    while (top < p.B) top *= 2;
    for (long long at = static_cast<long long>(blockIdx.x) * kPlanThreads + tid; at < items; at += step) {
        const int i = static_cast<int>(at);
        // the requests of token i, of taken page i and of given-back page i: how many sums are i at most
        int bt = 0, bp = 0, bb = 0;
        if (i < max(max(tokens, takes), backs))
            for (int s = top; s; s >>= 1) {
                if (bt + s <= p.B && tok_end[bt + s - 1] <= i) bt += s;
                if (bp + s <= p.B && take_end[bp + s - 1] <= i) bp += s;
                if (bb + s <= p.B && back_end[bb + s - 1] <= i) bb += s;
            }
        const int *id = nullptr, *taken = nullptr, *back = nullptr;
        int* to = nullptr;
        unsigned pos = 0, in = 0;
        if (i < tokens) {
            pos = held[bt] + i - (bt ? tok_end[bt - 1] : 0);
            const unsigned n = over_page(pos), have = pages_for(held[bt]);
            in = pos - n * page;
            id = n < have ? p.table + bt * p.ldt + n : p.ring + in_ring(head + (bt ? take_end[bt - 1] : 0) + n - have);
        }
        if (i < takes) {
            taken = p.ring + in_ring(static_cast<unsigned>(head) + i);
            to = p.table + bp * p.ldt + pages_for(held[bp]) + i - (bp ? take_end[bp - 1] : 0);
        }
        if (i < backs) back = p.table + bb * p.ldt + i - (bb ? back_end[bb - 1] : 0);
        const int page_id = id ? __ldcg(id) : 0, taken_id = taken ? __ldcg(taken) : 0, back_id = back ? __ldcg(back) : 0;
        if (i < p.cap) {
            p.slots[i] = id ? page_id * p.page + static_cast<int>(in) : -1;
            p.positions[i] = pos;
        }
        if (taken) *to = taken_id;
        if (back) p.ring[in_ring(tail + i)] = back_id;
        if (i <= p.B) p.starts[i] = go && i ? tok_end[i - 1] : 0;
    }

    // in place: when every CTA is past its reads
    if (p.in_place) {
        __syncthreads();
        if (gridDim.x > 1) {
            if (tid == 0) {
                const bool last = ptx::atom_add_acq_rel_gpu(p.counter, 1) == static_cast<int>(gridDim.x) - 1;
                if (last) ptx::st_relaxed_gpu(p.counter, 0);
                s_last = last;
            }
            __syncthreads();
            if (!s_last) return;
        }
        if (go)
            for (int b = tid; b < p.B; b += kPlanThreads) {
                const int ended = back_end[b] - (b ? back_end[b - 1] : 0), more = tok_end[b] - (b ? tok_end[b - 1] : 0);
                p.length_out[b] = ended ? 0 : held[b] + more;
            }
        else if (p.length_out != p.length)
            for (int b = tid; b < p.B; b += kPlanThreads) p.length_out[b] = held[b];
    } else if (blockIdx.x) {
        return;
    }
    if (tid == 0) {
        p.state_out[0] = go ? in_ring(static_cast<unsigned>(head) + takes) : head;
        p.state_out[1] = free - takes + backs;
        p.state_out[2] = tokens;
        p.state_out[3] = lacking;
    }
}

template <int kPlanThreads>
cudaError_t launch(const PagePlanParams& p, int num_sms, cudaStream_t stream, bool pdl)
{
    // (the pages that ended requests give back are not known here: room for a few of each)
    const long long items = p.cap > 8 * p.B ? p.cap : 8 * p.B, want = (items + kPlanThreads - 1) / kPlanThreads;
    const int grid = want < 1 ? 1 : want < num_sms ? static_cast<int>(want) : num_sms;
    return launch_grid(page_plan_kernel<kPlanThreads>, p, grid, kPlanThreads, 16 * p.B, stream, false, pdl);
}

}  // namespace

cudaError_t prepare_page_plan()
{
    return cudaFuncSetAttribute(page_plan_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * kMaxRequests);
}

// Threads of a CTA: one for each request, where there are many a few, so that sums and
// barriers are short.  256 / 512 / 1024 threads, us: 256 requests 3.6 / 4.0 / 5.2, 1024 4.8
// / 4.5 / 5.7, 4096 14.3 / 9.5 / 8.4.
cudaError_t launch_page_plan(const PagePlanParams& p, int num_sms, cudaStream_t stream, bool pdl)
{
    if (p.B <= 256) return launch<256>(p, num_sms, stream, pdl);
    if (p.B <= 2048) return launch<512>(p, num_sms, stream, pdl);
    return launch<1024>(p, num_sms, stream, pdl);
}

}  // namespace tovl
