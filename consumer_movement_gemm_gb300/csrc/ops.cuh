// ops.cuh -- parameter blocks and launchers of the decode-step operators:
// residual + RMS norm, router top-k, the expert layer for few tokens, products
// with 4-bit weights.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include "ctrl.cuh"

namespace tovl {

constexpr int kMaxDecodeRows = 64;     // tokens of one moe_decode / matvec_q4 call
constexpr int kMaxDecodeK = 16;        // experts per token of one moe_decode call
constexpr int kMaxTopk = 32;           // experts per token of one route_topk call
constexpr int kXScaleGroup = 128;      // columns per scale of 8-bit activations

// Counters of the streamed products (handle-owned, zero between calls), each
// of the first six in a 128-byte line of its own: tickets of up to two
// products, arrivals of three grid barriers, CTAs past the last one.
constexpr int kMaxGrid = 160;
constexpr int kSyncStep = 32;
constexpr int kTicketWord = 0;         // tickets of product i at word i * kTicketStep
constexpr int kBarrierWord = 2 * kSyncStep;
constexpr int kExitWord = 5 * kSyncStep;
constexpr int kPartWord = 6 * kSyncStep;                 // arrivals at a cut tile, by its first item (matvec_q4)
constexpr int kAttnWord = kPartWord + kMaxGrid * 8;      // arrivals at a shared segment, by its first CTA (attn_decode)
constexpr int kPagePlanWord = kAttnWord + 24 * kMaxGrid; // CTAs past their reads (page_plan)
constexpr int kSyncWords = kPagePlanWord + kSyncStep;

struct NormParams {
    const void* x;          // bf16 [T][H], rows ldx elements apart
    const void* residual;   // bf16 or fp32 [T][H], rows ldr apart; null = none
    void* residual_out;     // same type and stride
    const void* weight;     // bf16 [H]
    void* out;              // bf16 [T][H] rows ldo apart; null = none
    uint8_t* q;             // e4m3 [T][H] contiguous; null = none
    float* q_scale;         // [T][n_groups]
    long long ldx, ldr, ldo;
    float eps;
    int T, H;
    int group;              // columns per scale (H for one per row)
    int n_groups;
    int residual_f32;
};
cudaError_t launch_norm(const NormParams& p, int width, bool same_offset, int num_sms, cudaStream_t stream, bool pdl);

struct RouteParams {
    const void* logits;     // [T][E] fp32 or bf16, rows ld elements apart
    int* topk;              // [T][k]
    float* gate_w;          // [T][k]
    long long ld;
    int T, E, k;
    int f32;
    int renormalize;
};
cudaError_t launch_route(const RouteParams& p, cudaStream_t stream, bool pdl);

// One weight matrix (or one per expert): bf16 [E][K][N], or packed nibbles
// [E][K/8][N] with scales and zeros [E][K/group][N].
struct WeightMaps {
    CUtensorMap w, scale, zero;
};

// The same as addresses.
struct MoeWeights {
    const void* w;
    const void* scale;
    const void* zero;
};

// A call of the expert layer; the small form, whose time can be the host's, takes
// no more (a launch copies its parameters).
struct MoeCall {
    const void* x;          // bf16 [T][H], rows ldx apart
    long long ldx;
    const int* topk;        // [T][k]
    const float* gate_w;    // [T][k]
    void* out;              // bf16 [T][H], rows ldo apart
    long long ldo;
    void* h_hi;             // activations between the two products [T*k][I]: bf16, and
    void* h_lo;             // what the rounding left over; 4-bit weights: fp16, and its scales;
                            // small form: fp32 from h_hi on
    int T, k, E, H, I;
    Ctrl ctrl;
};

struct MoeDirectParams : MoeCall {
    MoeWeights up, down;    // W13, W2
};

struct MoeParams : MoeCall {
    WeightMaps w13, w2;
    int out_vec;            // rows of out allow 8-byte stores
    int most_parts;         // a tile is cut into most_parts + 2 parts at most
    float* part;            // [most_parts + 2][T*k][2I or H] parts of the products
    int* sync;              // kSyncWords counters
    int ready_offset;       // fault injection: CTAs that never come
    long long timeout_ns, pipe_timeout_ns;
};
// Expert layers without rings and barriers (moe_direct.cu), by the weights of the
// experts that the tokens can name, counted once per 16 tokens: up to 8 tokens
// fewer than 2^27 (bf16) or 2^26 (4-bit), more tokens fewer than 2^25.  Many small
// experts share those weights out to more CTAs with shorter sums, so the limit is
// lower for them.  Direct and through the rings, bf16 / 4-bit, us:
//   1 token, 2 of 8 experts of 256 x 128 (0.2M)       5.2 / 5.0     14.4 / 16.5
//   1 token, 2 of 8 of 4096 x 2048 (48M)             23.7 / 15.8    30.7 / 20.0
//   1 token, 2 of 8 of 4096 x 4096 (96M)             39.9 / 27.1    43.9 / 24.9
//   2 tokens, 2 of 8 of 4096 x 2048 (96M)            36.1 / 26.9    34.7 / 24.5
//   4 tokens, 2 of 8 of 4096 x 1024 (96M)            32.4 / 21.6    33.4 / 24.7
//   1 token, 4 of 8 of 4096 x 4096 (192M)            74.6 / 47.2    71.0 / 34.5
// 16 experts and more, bf16, up to 8 tokens: 2^26
//   2 tokens, 8 of 64 of 1024 x 512 (24M)            18.0 / 13.1    21.6 / 17.8
//   4 tokens, 4 of 32 of 1024 x 1024 (48M)           28.0 / 18.0    26.7 / 19.6
//   8 tokens, 4 of 32 of 1024 x 512 (48M)            26.6 / 17.7    24.8 / 19.5
//   4 tokens, 4 of 32 of 2048 x 1024 (96M)           40.6 / 27.0    34.8 / 25.0
//   8 tokens, 4 of 32 of 1024 x 1024 (96M)           39.0 / 29.2    32.6 / 24.9
// 64 (4-bit: 128): half of that
//   8 tokens, 8 of 64 of 512 x 256 (24M)             20.6 / 15.7    20.8 / 18.2
//   8 tokens, 16 of 128 of 512 x 256 (48M)           35.2 / 27.6    25.8 / 21.2
//   8 tokens, 8 of 64 of 1024 x 512 (96M)            41.4 / 29.7    34.3 / 25.6
// more than 8 tokens: 2^25
//   12 tokens, 2 of 8 of 512 x 256 (3M)               8.9 / 7.7     18.7 / 18.1
//   32 tokens, 2 of 8 of 1024 x 512 (24M)            18.8 / 15.8    20.0 / 20.4
//   33 tokens, 2 of 16 of 512 x 256 (18M)            14.9 / 13.7    17.2 / 19.1
//   32 tokens, 2 of 16 of 768 x 512 (36M)            26.3 / 23.7    20.9 / 18.4
//   64 tokens, 2 of 8 of 1024 x 512 (48M)            28.6 / 24.2    23.0 / 21.9
// more than 8 tokens, 64 (4-bit: 128) experts and more, counted once per 16 tokens: 2^24
//   20 tokens, 8 of 64 of 256 x 128 (12M)            18.7 / 15.8    17.6 / 18.7
//   64 tokens, 4 of 32 of 256 x 128 (12M)            16.5 / 16.7    17.8 / 20.3
//   48 tokens, 8 of 64 of 256 x 128 (18M)            24.5 / 23.9    19.7 / 21.4
//   20 tokens, 4 of 32 of 512 x 256 (24M)            22.0 / 16.2    17.9 / 18.1
//   16 tokens, 8 of 64 of 512 x 256 (24M)            31.1 / 22.4    22.3 / 18.8
//   64 tokens, 8 of 64 of 256 x 128 (24M)            27.2 / 28.9    21.1 / 22.2
inline bool use_direct_moe(int T, int k, int E, int H, int I, int group)
{
    const int most = T <= 8 ? 8 : 16, names = (T < most ? T : most) * k;
    const int experts = (T + most - 1) / most * (names < E ? names : E);
    const int log = (T > 8 ? 25 : group ? 26 : experts < 16 ? 27 : 26) - (experts >= (group ? 128 : 64) ? 1 : 0);
    return 3LL * experts * H * I < 1LL << log;
}
cudaError_t prepare_moe_direct();
cudaError_t launch_moe_direct(const MoeDirectParams& p, int group, bool zero, int sms, cudaStream_t stream, bool pdl);
cudaError_t prepare_moe_decode();
// group: rows per scale of 4-bit weights, 0 for bf16
cudaError_t launch_moe_decode(const MoeParams& p, int group, bool zero, int grid, cudaStream_t stream, bool cooperative,
                              bool pdl);

// 4-bit products that read the matrix straight into registers: those of fewer
// than 2^26 weights, counted once per 16 rows.  So and through the ring, one row
// and 16, us: below it, 4096 x 4096 4.9 / 7.1 and 8.4 / 15.6, 4096 x 11008 11.0 /
// 18.5 and 14.3 / 21.3; at the edge, 8192 x 8192 14.6 / 24.0 and 13.7 / 20.8; above
// it, 8192 x 28672 39 and 30.4.
inline bool use_direct(int T, int K, int N) { return static_cast<long long>((T + 15) / 16) * K * N < (1LL << 26); }

struct MatvecCall {
    const void* x;          // bf16 or e4m3 [T][K], rows ldx apart
    const float* x_scale;   // [T][ceil(K/128)] for e4m3
    void* out;              // bf16 [T][N], rows ldo apart
    long long ldx, ldo;
    int T, K, N;
};

struct MatvecDirectParams : MatvecCall {
    const void* wq;
    const void* w_scale;
    const void* w_zero;
};

struct MatvecParams : MatvecCall {
    WeightMaps w;
    float* part;            // [most_parts + 2][T][N] parts of the product
    int out_vec;            // rows of out allow 8-byte stores
    int most_parts;
    int* sync;
    long long timeout_ns, pipe_timeout_ns;
    Ctrl ctrl;
};
cudaError_t launch_matvec_q4_direct(const MatvecDirectParams& p, bool e4m3, int group, bool zero, int sms, cudaStream_t stream,
                                    bool pdl);
cudaError_t prepare_matvec_q4();
cudaError_t launch_matvec_q4(const MatvecParams& p, bool e4m3, int group, bool zero, int grid, cudaStream_t stream,
                             bool pdl);

// One persistent grid whose CTAs meet at barriers.
template <class Kernel, class Params>
cudaError_t launch_grid(Kernel kernel, const Params& p, int grid, int threads, int smem, cudaStream_t stream, bool cooperative,
                        bool pdl)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = cooperative ? 1 : 0;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

struct QuantParams {
    const void* w;          // bf16 [E][K][N]
    uint32_t* q;            // [E][K/8][N]
    void* scale;            // bf16 [E][K/group][N]
    uint8_t* zero;          // [E][K/group][N]; null = symmetric (zero 8)
    int E, K, N, group;
};
cudaError_t launch_quantize_q4(const QuantParams& p, cudaStream_t stream);

}  // namespace tovl
