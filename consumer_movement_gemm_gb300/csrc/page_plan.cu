// page_plan.cu -- pages, cache slots and positions of a step's new tokens.
//
// Every CTA scans all requests' counts for itself (prefix sums of new tokens,
// of pages taken and of pages given back, in shared memory) and works on a
// share of the outputs: a token or a page finds its request by bisection.
// Pages are taken from the ring's head in the order of the requests, so a
// token's page is known from the sums alone and nothing waits for the table.
// Given-back pages go behind the ring's tail, which no taken page lies at.
// What may be updated in place (lengths, state) is written by the CTA that
// finishes last, when all others have read it.
//
// What bounds it: latency (a launch, the dependent loads of counts, ring and
// table), then the bisections of long prompts.
#include "common.cuh"
#include "paged.cuh"
#include "sync.cuh"

namespace tovl {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kTokensPerCta = 2048;

// First of n ascending sums that is over i.
__device__ __forceinline__ int request_of(const int* sum, int n, int i)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] > i) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlanParams p)
{
    extern __shared__ int sums[];          // inclusive: tokens, pages taken, pages given back
    __shared__ long long s_warp[3][kPlanWarps];
    __shared__ int s_last;
    int* const tok_end = sums;
    int* const take_end = sums + p.B;
    int* const back_end = sums + 2 * p.B;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    const int per = (p.B + kPlanThreads - 1) / kPlanThreads, b0 = tid * per, b1 = min(p.B, b0 + per);
    const int head = __ldcg(p.state), free = __ldcg(p.state + 1);
    const auto pages_for = [&](long long tokens) { return static_cast<int>((tokens + p.page - 1) / p.page); };
    const long long most = static_cast<long long>(p.width) * p.page;
    long long sum[3] = {0, 0, 0};
    bool bad = head < 0 || head >= p.pages || free < 0 || free > p.pages;
    for (int b = b0; b < b1; ++b) {
        const int len = __ldcg(p.length + b), add = __ldcg(p.add + b);
        if (len < 0 || add < -1 || static_cast<long long>(len) + max(add, 0) > most) {
            bad = true;
            continue;
        }
        const int have = pages_for(len);
        sum[0] += max(add, 0);
        sum[1] += add > 0 ? pages_for(static_cast<long long>(len) + add) - have : 0;
        sum[2] += add < 0 ? have : 0;
    }
    long long before[3], total[3] = {0, 0, 0};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        before[k] = sum[k];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long o = __shfl_up_sync(0xffffffffu, before[k], d);
            if (lane >= d) before[k] += o;
        }
        if (lane == 31) s_warp[k][warp] = before[k];
        before[k] -= sum[k];
    }
    bad = __syncthreads_or(bad);
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            if (w < warp) before[k] += s_warp[k][w];
            total[k] += s_warp[k][w];
        }
    bad = bad || total[0] > p.cap || free + total[2] > p.pages;
    const int lacking = bad ? -1 : total[1] > free ? static_cast<int>(total[1] - free) : 0;
    const bool go = lacking == 0;
    if (go) {
        int run[3] = {static_cast<int>(before[0]), static_cast<int>(before[1]), static_cast<int>(before[2])};
        for (int b = b0; b < b1; ++b) {
            const int len = __ldcg(p.length + b), add = __ldcg(p.add + b), have = pages_for(len);
            run[0] += max(add, 0);
            run[1] += add > 0 ? pages_for(static_cast<long long>(len) + add) - have : 0;
            run[2] += add < 0 ? have : 0;
            tok_end[b] = run[0], take_end[b] = run[1], back_end[b] = run[2];
        }
    } else if (bad && blockIdx.x == 0 && tid == 0) {
        record_error(p.ctrl, kErrInvalid);
    }
    __syncthreads();

    const int at = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
    const int tokens = go ? static_cast<int>(total[0]) : 0, takes = go ? static_cast<int>(total[1]) : 0;
    const int backs = go ? static_cast<int>(total[2]) : 0;
    const auto ring_at = [&](long long i) { return i >= p.pages ? static_cast<int>(i - p.pages) : static_cast<int>(i); };
    for (long long i = at; i < p.cap; i += step) {
        int slot = -1, pos = 0;
        if (i < tokens) {
            const int b = request_of(tok_end, p.B, static_cast<int>(i));
            const int len = __ldcg(p.length + b), have = pages_for(len);
            pos = len + static_cast<int>(i) - (b ? tok_end[b - 1] : 0);
            const int n = pos / p.page, in = pos - n * p.page;
            const int id = n < have ? __ldcg(p.table + b * p.ldt + n)
                                    : __ldcg(p.ring + ring_at(static_cast<long long>(head) + (b ? take_end[b - 1] : 0) + n - have));
            slot = id * p.page + in;
        }
        p.slots[i] = slot;
        p.positions[i] = pos;
    }
    for (long long j = at; j < takes; j += step) {
        const int b = request_of(take_end, p.B, static_cast<int>(j));
        const int have = pages_for(__ldcg(p.length + b));
        p.table[b * p.ldt + have + j - (b ? take_end[b - 1] : 0)] = __ldcg(p.ring + ring_at(head + j));
    }
    for (long long j = at; j < backs; j += step) {
        const int b = request_of(back_end, p.B, static_cast<int>(j));
        p.ring[ring_at(ring_at(static_cast<long long>(head) + free) + j)] =
            __ldcg(p.table + b * p.ldt + j - (b ? back_end[b - 1] : 0));
    }
    for (int b = at; b <= p.B; b += step) p.starts[b] = go && b ? tok_end[b - 1] : 0;

    // in place: when every CTA is past its reads
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
    for (int b = tid; b < p.B; b += kPlanThreads) {
        const int len = __ldcg(p.length + b), add = __ldcg(p.add + b);
        p.length_out[b] = !go ? len : add < 0 ? 0 : len + add;
    }
    if (tid == 0) {
        p.state_out[0] = go ? ring_at(static_cast<long long>(head) + takes) : head;
        p.state_out[1] = free - takes + backs;
        p.state_out[2] = tokens;
        p.state_out[3] = lacking;
    }
}

}  // namespace

cudaError_t prepare_page_plan()
{
    return cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * 4 * kMaxRequests);
}

cudaError_t launch_page_plan(const PagePlanParams& p, int num_sms, cudaStream_t stream, bool pdl)
{
    const long long want = (static_cast<long long>(p.cap) + kTokensPerCta - 1) / kTokensPerCta;
    const int grid = want < 1 ? 1 : want < num_sms ? static_cast<int>(want) : num_sms;
    return launch_grid(page_plan_kernel, p, grid, kPlanThreads, 3 * 4 * p.B, stream, false, pdl);
}

}  // namespace tovl
