// ops_api.cu -- host side of the decode-step operators declared in
// include/tovl.h: argument checks, tensor maps, launches.  None of them is a
// protocol round (the handle's sequence number stays).
#include <cstring>
#include "ctx.cuh"
#include "ops.cuh"

namespace {

// A map of stacked [rows][width] matrices; boxes of box_inner columns x
// box_rows rows, out-of-range elements read as zero.
int encode_3d(tovl_ctx* h, CUtensorMap* map, CUtensorMapDataType type, int elem, const void* base, uint64_t width,
              uint64_t rows, uint64_t outer, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    cuuint64_t dims[3] = {width, rows, outer};
    cuuint64_t strides[2] = {width * elem, width * elem * rows};
    cuuint32_t box[3] = {box_inner, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = h->encode(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(h->last_error, sizeof h->last_error, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
        return TOVL_ERR_INVALID;
    }
    return TOVL_OK;
}

// Blocks of one warp: 64 columns x 32 rows of bf16, 32 columns x 256 rows of 4 bits.
int map_bf16(tovl_ctx* h, WeightMaps* m, const void* w, int E, int K, int N)
{
    return encode_3d(h, &m->w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, w, N, K, E, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
}

int map_q4(tovl_ctx* h, WeightMaps* m, const void* q, const void* scale, const void* zero, int E, int K, int N, int group)
{
    int rc = encode_3d(h, &m->w, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, q, N, K / 8, E, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc == TOVL_OK)
        rc = encode_3d(h, &m->scale, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, scale, N, K / group, E, 32, 256 / group,
                       CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc == TOVL_OK && zero)
        rc = encode_3d(h, &m->zero, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, zero, N, K / group, E, 32, 256 / group,
                       CU_TENSOR_MAP_SWIZZLE_NONE);
    return rc;
}

bool valid_group(int group)
{
    return group == 32 || group == 64 || group == 128;
}

// Shape of one packed matrix: whole groups, rows of 16 bytes (of 16 zeros).
bool valid_q4(int K, int N, int group, const void* q, const void* scale, const void* zero)
{
    return K % group == 0 && N % (zero ? 16 : 8) == 0 && q && scale && aligned16(q) && aligned16(scale) && aligned16(zero);
}

long long up256(long long v) { return (v + 255) & ~255LL; }

// Limit of a tile's parts (less two) by the rows of a product and its tiles of
// 512 columns: few rows and few tiles can afford a cut for every CTA, many have
// other tiles to share out.
int most_parts(long long rows, long long N)
{
    const int by_rows = rows <= 64 ? 16 : rows <= 256 ? 8 : 4, by_tiles = N < 64 * 512 ? 16 : N < 256 * 512 ? 8 : 4;
    return by_rows < by_tiles ? by_rows : by_tiles;
}

// Pieces of a moe_decode workspace, in order.
struct MoeSpace {
    long long h, part, total;
    MoeSpace(int T, int k, int H, int I)
    {
        const long long rows = static_cast<long long>(T) * k;
        h = up256(2 * rows * I);
        part = 4 * (most_parts(rows, 0) + 2) * rows * (2 * I > H ? 2 * I : H);
        total = 2 * h + up256(part);
    }
};

bool valid_moe_shape(int T, int k, int H, int I)
{
    return T >= 0 && k >= 1 && H >= 8 && I >= 8 && H % 8 == 0 && I % 8 == 0;
}

bool fits_moe(int T, int k, int H, int I)
{
    return T <= kMaxDecodeRows && k <= kMaxDecodeK && H <= kMaxK && I <= kMaxK;
}

}  // namespace

TOVL_API int tovl_add_rmsnorm(tovl_handle h, const void* x, long long ldx, const void* residual, void* residual_out,
                              int residual_type, long long ldr, const void* weight, float eps, int T, int H, void* out,
                              long long ldo, void* q, float* q_scale, int group, void* stream)
{
    if (!h) return TOVL_ERR_INVALID;
    if (T < 0 || H < 1 || (!out && !q) || (q && !q_scale) || !(eps >= 0.f)) return TOVL_ERR_INVALID;
    if (H > kMaxK) return TOVL_ERR_UNSUPPORTED;
    if (residual && (!residual_out || (residual_type != TOVL_BF16 && residual_type != TOVL_F32))) return TOVL_ERR_INVALID;
    if (q && group != 0 && !valid_group(group)) return TOVL_ERR_UNSUPPORTED;
    if (T == 0) return TOVL_OK;
    if (!x || !weight || ldx < H || (residual && ldr < H) || (out && ldo < H)) return TOVL_ERR_INVALID;
    const int res_size = residual_type == TOVL_F32 ? 4 : 2;
    if (!aligned(x, 2) || !aligned(weight, 2) || !aligned(out, 2) || !aligned(q_scale, 4) ||
        (residual && (!aligned(residual, res_size) || !aligned(residual_out, res_size))))
        return TOVL_ERR_INVALID;
    NormParams p = {};
    p.x = x;
    p.weight = weight;
    p.out = out;
    p.q = static_cast<uint8_t*>(q);
    p.q_scale = q_scale;
    p.ldx = ldx;
    p.ldo = ldo;
    p.eps = eps;
    p.T = T;
    p.H = H;
    p.group = group ? group : H;
    p.n_groups = static_cast<int>(ceil_div(H, p.group));
    if (residual) {
        p.residual = residual;
        p.residual_out = residual_out;
        p.ldr = ldr;
        p.residual_f32 = residual_type == TOVL_F32;
    }
    // the widest accesses that every row start allows: 16 bytes, pairs, single elements
    const auto fits = [&](int w) {
        return H % w == 0 && ldx % w == 0 && aligned(x, 2 * w) && aligned(weight, 2 * w) &&
               (!out || (ldo % w == 0 && aligned(out, 2 * w))) && (!q || aligned(q, w)) &&
               (!residual || (ldr % w == 0 && aligned(residual, w == 8 ? 16 : res_size * w) &&
                              aligned(residual_out, w == 8 ? 16 : res_size * w)));
    };
    const int width = fits(8) ? 8 : fits(2) ? 2 : 1;
    // every tensor's rows start at the same distance from a 16-byte boundary (8 bytes of e4m3)
    const auto offset = [](const void* ptr, int size, int piece) { return static_cast<int>(reinterpret_cast<uintptr_t>(ptr) / size) & (piece - 1); };
    const int off = offset(x, 2, 8), piece = res_size == 4 ? 4 : 8;
    const auto like_x = [&](const void* ptr, long long ld, int size, int n) { return (T == 1 || (ld - ldx) % n == 0) && offset(ptr, size, n) == (off & (n - 1)); };
    const bool same_offset = aligned16(weight) && (!out || like_x(out, ldo, 2, 8)) && (!q || like_x(q, H, 1, 8)) &&
                             (!residual || (like_x(residual, ldr, res_size, piece) && like_x(residual_out, ldr, res_size, piece)));
    DeviceGuard g(h->device);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return run(h, s, "norm launch", [&](bool pdl) { return launch_norm(p, width, same_offset, h->num_sms, s, pdl); });
}

TOVL_API int tovl_route_topk(tovl_handle h, const void* logits, int type, long long ld, int T, int E, int k,
                             int renormalize, int* topk_idx, float* gate_w, void* stream)
{
    if (!h) return TOVL_ERR_INVALID;
    if (T < 0 || E < 1 || k < 1 || (type != TOVL_BF16 && type != TOVL_F32)) return TOVL_ERR_INVALID;
    if (E > kMaxExperts || k > kMaxTopk) return TOVL_ERR_UNSUPPORTED;
    if (T == 0) return TOVL_OK;
    if (!logits || !topk_idx || !gate_w || ld < E || !aligned(logits, type == TOVL_F32 ? 4 : 2) || !aligned(topk_idx, 4) ||
        !aligned(gate_w, 4))
        return TOVL_ERR_INVALID;
    RouteParams p = {};
    p.logits = logits;
    p.topk = topk_idx;
    p.gate_w = gate_w;
    p.ld = ld;
    p.T = T;
    p.E = E;
    p.k = k;
    p.f32 = type == TOVL_F32;
    p.renormalize = renormalize != 0;
    DeviceGuard g(h->device);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return run(h, s, "route launch", [&](bool pdl) { return launch_route(p, s, pdl); });
}

TOVL_API long long tovl_moe_decode_workspace(tovl_handle h, int T, int k, int H, int I)
{
    if (!h || !valid_moe_shape(T, k, H, I) || !fits_moe(T, k, H, I)) return -1;
    return MoeSpace(T, k, H, I).total;
}

// The part that both weight types share.  group: rows per scale, 0 for bf16.
static int run_moe(tovl_handle h, const MoeWeights& up, const MoeWeights& down, int group, const void* x, long long ldx, int T, int H,
                   const int* topk_idx, const float* gate_w, int k, int E, int I, void* out, long long ldo, void* workspace,
                   long long workspace_bytes, void* stream)
{
    if (!x || !topk_idx || !gate_w || !out || !workspace || ldx < H || ldo < H || ldx % 8 || !aligned16(x) ||
        !aligned(out, 2) || !aligned(topk_idx, 4) || !aligned(gate_w, 4) || !aligned(workspace, 256))
        return TOVL_ERR_INVALID;
    const MoeSpace space(T, k, H, I);
    if (workspace_bytes < space.total) return TOVL_ERR_INVALID;
    DeviceGuard g(h->device);
    const bool zero = up.zero != nullptr;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    MoeCall c = {};
    c.x = x;
    c.ldx = ldx;
    c.topk = topk_idx;
    c.gate_w = gate_w;
    c.out = out;
    c.ldo = ldo;
    c.h_hi = ws;
    c.h_lo = ws + space.h;
    c.T = T;
    c.k = k;
    c.E = E;
    c.H = H;
    c.I = I;
    c.ctrl = h->ctrl;
    // (an injected fault is a barrier's, which the small form does not have)
    if (!h->fault_gate_offset && use_direct_moe(T, k, E, H, I, group)) {
        MoeDirectParams p = {c, up, down};
        return run(h, s, "expert layer launch", [&](bool pdl) { return launch_moe_direct(p, group, zero, h->num_sms, s, pdl); });
    }
    MoeParams p;
    std::memset(&p, 0, sizeof p);
    static_cast<MoeCall&>(p) = c;
    int rc = group ? map_q4(h, &p.w13, up.w, up.scale, up.zero, E, H, 2 * I, group) : map_bf16(h, &p.w13, up.w, E, H, 2 * I);
    if (rc == TOVL_OK)
        rc = group ? map_q4(h, &p.w2, down.w, down.scale, down.zero, E, I, H, group) : map_bf16(h, &p.w2, down.w, E, I, H);
    if (rc != TOVL_OK) return rc;
    p.out_vec = ldo % 4 == 0 && aligned(out, 8);
    p.most_parts = most_parts(static_cast<long long>(T) * k, 0);
    p.part = reinterpret_cast<float*>(ws + 2 * space.h);
    p.sync = h->sync_words;
    p.ready_offset = h->fault_gate_offset;
    p.timeout_ns = h->timeout_ns;
    p.pipe_timeout_ns = 4 * h->timeout_ns + 100000000LL;
    return run(h, s, "expert layer launch",
               [&](bool pdl) { return launch_moe_decode(p, group, zero, h->num_sms, s, h->coop_enabled, pdl); });
}

TOVL_API int tovl_moe_decode(tovl_handle h, const void* x, long long ldx, int T, int H, const int* topk_idx,
                             const float* gate_w, int k, int E, const void* W13, const void* W2, int I, void* out,
                             long long ldo, void* workspace, long long workspace_bytes, void* stream)
{
    if (!h) return TOVL_ERR_INVALID;
    if (!valid_moe_shape(T, k, H, I) || E < 1 || !W13 || !W2 || !aligned16(W13) || !aligned16(W2)) return TOVL_ERR_INVALID;
    if (!fits_moe(T, k, H, I) || E > kMaxExperts || h->num_sms > kMaxGrid) return TOVL_ERR_UNSUPPORTED;
    if (T == 0) return TOVL_OK;
    return run_moe(h, {W13, nullptr, nullptr}, {W2, nullptr, nullptr}, 0, x, ldx, T, H, topk_idx, gate_w, k, E, I, out, ldo, workspace,
                   workspace_bytes, stream);
}

TOVL_API int tovl_moe_decode_q4(tovl_handle h, const void* x, long long ldx, int T, int H, const int* topk_idx,
                                const float* gate_w, int k, int E, const void* W13_q, const void* W13_scale,
                                const void* W13_zero, const void* W2_q, const void* W2_scale, const void* W2_zero,
                                int group, int I, void* out, long long ldo, void* workspace, long long workspace_bytes,
                                void* stream)
{
    if (!h) return TOVL_ERR_INVALID;
    if (!valid_moe_shape(T, k, H, I) || E < 1 || (!W13_zero) != (!W2_zero)) return TOVL_ERR_INVALID;
    if (!valid_group(group)) return TOVL_ERR_UNSUPPORTED;
    if (!valid_q4(H, 2 * I, group, W13_q, W13_scale, W13_zero) || !valid_q4(I, H, group, W2_q, W2_scale, W2_zero))
        return TOVL_ERR_INVALID;
    if (!fits_moe(T, k, H, I) || E > kMaxExperts || h->num_sms > kMaxGrid) return TOVL_ERR_UNSUPPORTED;
    if (T == 0) return TOVL_OK;
    return run_moe(h, {W13_q, W13_scale, W13_zero}, {W2_q, W2_scale, W2_zero}, group, x, ldx, T, H, topk_idx, gate_w, k, E, I, out, ldo,
                   workspace, workspace_bytes, stream);
}

TOVL_API long long tovl_matvec_q4_workspace(tovl_handle h, int T, int N)
{
    if (!h || T < 0 || N < 1 || T > kMaxDecodeRows) return -1;
    return up256(4LL * (most_parts(T, N) + 2) * T * N);
}

TOVL_API int tovl_matvec_q4(tovl_handle h, const void* x, int x_type, const float* x_scale, long long ldx, int T, int K,
                            const void* wq, const void* w_scale, const void* w_zero, int group, int N, void* out,
                            long long ldo, void* workspace, long long workspace_bytes, void* stream)
{
    if (!h) return TOVL_ERR_INVALID;
    if (T < 0 || K < 1 || N < 1 || (x_type != TOVL_BF16 && x_type != TOVL_E4M3) || (x_type == TOVL_E4M3 && !x_scale))
        return TOVL_ERR_INVALID;
    if (!valid_group(group)) return TOVL_ERR_UNSUPPORTED;
    if (!valid_q4(K, N, group, wq, w_scale, w_zero)) return TOVL_ERR_INVALID;
    if (T > kMaxDecodeRows || K > kMaxK || N > (1 << 24) || h->num_sms > kMaxGrid) return TOVL_ERR_UNSUPPORTED;
    if (T == 0) return TOVL_OK;
    const int row = x_type == TOVL_BF16 ? 8 : 16;      // elements that 16 bytes hold
    if (!x || !out || !workspace || ldx < K || ldo < N || ldx % row || !aligned16(x) || !aligned(out, 2) ||
        !aligned(x_scale, 4) || !aligned(workspace, 256) || workspace_bytes < tovl_matvec_q4_workspace(h, T, N))
        return TOVL_ERR_INVALID;
    DeviceGuard g(h->device);
    const bool e4m3 = x_type == TOVL_E4M3, zero = w_zero != nullptr;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const MatvecCall c = {x, x_scale, out, ldx, ldo, T, K, N};
    if (use_direct(T, K, N)) {
        const MatvecDirectParams p = {c, wq, w_scale, w_zero};
        return run(h, s, "4-bit product launch",
                   [&](bool pdl) { return launch_matvec_q4_direct(p, e4m3, group, zero, h->num_sms, s, pdl); });
    }
    MatvecParams p;
    std::memset(&p, 0, sizeof p);
    static_cast<MatvecCall&>(p) = c;
    const int rc = map_q4(h, &p.w, wq, w_scale, w_zero, 1, K, N, group);
    if (rc != TOVL_OK) return rc;
    p.part = static_cast<float*>(workspace);
    p.out_vec = ldo % 4 == 0 && aligned(out, 8);
    p.most_parts = most_parts(T, N);
    p.sync = h->sync_words;
    p.timeout_ns = h->timeout_ns;
    p.pipe_timeout_ns = 4 * h->timeout_ns + 100000000LL;
    p.ctrl = h->ctrl;
    return run(h, s, "4-bit product launch",
               [&](bool pdl) { return launch_matvec_q4(p, e4m3, group, zero, h->num_sms, s, pdl); });
}

TOVL_API int tovl_quantize_q4(tovl_handle h, const void* W, int E, int K, int N, int group, void* wq, void* w_scale,
                              void* w_zero, void* stream)
{
    if (!h) return TOVL_ERR_INVALID;
    if (E < 1 || K < 1 || N < 1 || !W || !aligned(W, 2)) return TOVL_ERR_INVALID;
    if (!valid_group(group)) return TOVL_ERR_UNSUPPORTED;
    if (!valid_q4(K, N, group, wq, w_scale, w_zero)) return TOVL_ERR_INVALID;
    QuantParams p = {};
    p.w = W;
    p.q = static_cast<uint32_t*>(wq);
    p.scale = w_scale;
    p.zero = static_cast<uint8_t*>(w_zero);
    p.E = E;
    p.K = K;
    p.N = N;
    p.group = group;
    DeviceGuard g(h->device);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_quantize_q4(p, s);
    if (e != cudaSuccess) return cuda_fail(h, e, "quantise launch");
    h->last_stream = s;
    return TOVL_OK;
}
