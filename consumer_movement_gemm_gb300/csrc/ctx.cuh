// ctx.cuh -- the handle behind tovl_handle and the host helpers that the API
// translation units share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <cstdio>

#include "tovl.h"
#include "ctrl.cuh"

#define TOVL_API extern "C" __attribute__((visibility("default")))

using namespace tovl;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct tovl_ctx {
    tovl_config cfg;
    int device = 0;
    int num_sms = 0;
    int producers = 0;       // 0 = automatic split per call
    int last_P = 0, last_C = 0;
    int consumers = 0;
    int copy_mode = TOVL_COPY_AUTO;     // vector below 8 KB rows, bulk from 8 KB (measured best per size)
    int stats = 0;
    long long timeout_ns = 2000000000LL;
    int copy_ctas = 0;       // copy sweep copiers (0 = auto)
    int copy_waiters = 0;    // copy sweep waiters (0 = auto)
    int fault_gate_offset = 0;  // test hook: gates wait for seq + offset
    int slices = 1;          // K-slices per chunk watermark (fixed per handle)
    int pair_mode = 1;       // gather calls use CTA-pair (cta_group::2) consumers when possible
    int max_pairs = 0;       // co-resident CTA pairs of the pair kernel on this device
    bool coop_pairs = true;  // cooperative launch accepted together with clusters
    bool coop_enabled = true;  // fused launches ask for the co-residency guarantee
    int producer_mode = 0;     // fused producers: 0 vector copies, 1 staged bulk loads
    int dispatch_align = kBlockRows;  // expert segment alignment: 128, or 256 for CTA-pair tiles
    bool pdl = true;           // programmatic dependent launch between this library's kernels
    int role_switch = 1;       // 1: dispatch (single-CTA tiles) and reduce-scatter roles switch; 2: CTA-pair dispatch too
    int embedded = 1;          // without producer CTAs, the consumer CTAs' spare warps copy: 1 dispatch, 2 also gather
    int rs_epi = 0;            // 1: reduce-scatter tiles are summed by their owners' idle warps (no producer CTAs)
    int wide_tiles = 1;        // 1: CTA-pair dispatch tiles (embedded producers) are 256 x 512 where N allows
    int l2_hints = -1;         // kHint* bits for every fused call; -1 = each call's measured default
    bool pdl_ok = true;        // cleared if the device rejects the launch attribute
    long long seq = 0;
    Ctrl ctrl{};
    Plan plan{};
    int max_seg = 0;
    void* ctrl_mem = nullptr;    // one allocation for the control plane
    void* plan_mem = nullptr;    // one allocation for plan scratch
    cudaStream_t last_stream = nullptr;
    const void* last_dispatched = nullptr;
    int last_T = 0, last_k = 0, last_E = 0;
    long long last_tiles = 0;    // tiles and K-slices of the last fused call (trace layout)
    int last_ks = 0;
    EncodeTiledFn encode = nullptr;
    int* sync_words = nullptr;   // kSyncWords counters of the split-tile kernels; zero between calls
    char last_error[256] = {0};
};

inline int cuda_fail(tovl_ctx* h, cudaError_t e, const char* what)
{
    if (h) std::snprintf(h->last_error, sizeof h->last_error, "%s: %s", what, cudaGetErrorString(e));
    return TOVL_ERR_CUDA;
}

inline bool aligned16(const void* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

inline long long ceil_div(long long a, long long b)
{
    return (a + b - 1) / b;
}

struct DeviceGuard {
    int prev = 0;
    explicit DeviceGuard(int dev)
    {
        cudaGetDevice(&prev);
        if (prev != dev) cudaSetDevice(dev);
    }
    ~DeviceGuard() { cudaSetDevice(prev); }
};
