// paged_api.cu -- host side of the paged attention step declared in
// include/tovl.h: argument checks and launches.  None of the calls is a
// protocol round (the handle's sequence number stays).
#include <climits>
#include <cstring>
#include "ctx.cuh"
#include "paged.cuh"

namespace {

constexpr int kMaxQueryHeads = 4096;
constexpr int kMaxDecodeBatch = 65536;
constexpr int kMaxNewTokens = 1 << 30;

// log2(n), or -1
int shift_of(int n)
{
    for (int s = 0; s < 31; ++s)
        if (n == 1 << s) return s;
    return -1;
}

// The cache as the kernels take it.
int check_cache(const tovl_kv_cache* c, KvCache* out)
{
    if (!c || (c->type != TOVL_BF16 && c->type != TOVL_E4M3) || c->pages < 1 || c->page < 1 || c->heads < 1 || c->dim < 1)
        return TOVL_ERR_INVALID;
    const int size = c->type == TOVL_BF16 ? 2 : 1;
    if (c->dim > kMaxHeadDim || c->dim * size % 16 || c->heads > kMaxQueryHeads ||
        static_cast<long long>(c->pages) * c->page > INT_MAX)
        return TOVL_ERR_UNSUPPORTED;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return TOVL_ERR_INVALID;
    if (size == 1 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return TOVL_ERR_INVALID;
    const long long strides[3] = {c->page_stride, c->slot_stride, c->head_stride};
    const int extents[3] = {c->pages, c->page, c->heads};
    for (int i = 0; i < 3; ++i)
        if (extents[i] > 1 && (strides[i] < c->dim || strides[i] * size % 16)) return TOVL_ERR_INVALID;
    out->k = static_cast<uint8_t*>(c->k);
    out->v = static_cast<uint8_t*>(c->v);
    out->k_scale = c->k_scale;
    out->v_scale = c->v_scale;
    out->page_stride = c->pages > 1 ? c->page_stride * size : 0;
    out->slot_stride = c->page > 1 ? c->slot_stride * size : 0;
    out->head_stride = c->heads > 1 ? c->head_stride * size : 0;
    out->pages = c->pages;
    out->page = c->page;
    out->heads = c->heads;
    out->dim = c->dim;
    out->page_shift = shift_of(c->page);
    return TOVL_OK;
}

// Rows of whole 16-byte pieces.
bool valid_rows(const void* p, long long ld, long long width)
{
    return p && aligned16(p) && ld >= width && ld % 8 == 0;
}

// Maps of a cache's keys and values for boxes of `rows` slots, where the layout
// allows them: whole boxes of at least 8 slots in a page (1024 bytes of shared
// memory, the swizzle's period), strides that nest.  False: rows one by one, which
// is also faster for rows of one box that start off the 32-byte sectors.  64 requests
// of 4096 tokens, 4 heads for 16, boxes / rows, us: e4m3 of 16 50 / 33, of 48 50 / 39, of
// 80 61 / 48, of 112 60 / 58, bf16 of 40 53 / 44; rows of two boxes: bf16 of 72 67 / 67,
// e4m3 of 144 78 / 80; rows of whole sectors: e4m3 of 32 42 / 33 (the rule loses there), of
// 64 35 / 34, of 96 50 / 49, bf16 of 16 33 / 37, of 32 33 / 36, of 48 43 / 45.
bool map_cache(tovl_ctx* h, AttnParams* p, bool e4m3, const AttnShape& shape, int together)
{
    const int tile = shape.rows, box_bytes = shape.box_bytes;
    int rows = tile;
    while (rows > 1 && p->cache.page % rows) rows /= 2;
    const int row_bytes = p->cache.dim * (e4m3 ? 1 : 2);
    if (rows * box_bytes < 1024 || (row_bytes < 128 && row_bytes % 32)) return false;
    if (e4m3 && (!aligned16(p->cache.k_scale) || !aligned16(p->cache.v_scale))) return false;
    const int size = e4m3 ? 1 : 2;
    const KvCache& c = p->cache;
    const cuuint64_t row = row_bytes;
    // the dimension with the smaller stride first; extents of 1 take any
    p->slots_first = c.heads > 1 && c.page > 1 && c.slot_stride < c.head_stride;
    cuuint64_t n[2] = {static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.page)};
    cuuint64_t step[2] = {static_cast<cuuint64_t>(c.head_stride), static_cast<cuuint64_t>(c.slot_stride)};
    cuuint32_t in_box[2] = {1, static_cast<cuuint32_t>(rows)};
    const int a = p->slots_first ? 1 : 0, b = 1 - a;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), n[a], n[b], static_cast<cuuint64_t>(c.pages)};
    cuuint64_t strides[3] = {n[a] > 1 ? step[a] : row, 0, 0};
    strides[1] = n[b] > 1 ? step[b] : strides[0] * n[a];
    strides[2] = c.pages > 1 ? static_cast<cuuint64_t>(c.page_stride) : strides[1] * n[b];
    if (strides[1] % strides[0] || strides[2] % strides[1] || strides[2] >> 40) return false;
    cuuint32_t box[4] = {static_cast<cuuint32_t>(box_bytes / size), in_box[a], in_box[b], 1};
    cuuint32_t every[4] = {1, 1, 1, 1};
    const auto encode = [&](CUtensorMap* map, void* base) {
        return h->encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, every,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         together > 1 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (!encode(&p->k_map, c.k) || !encode(&p->v_map, c.v)) return false;
    while (rows << p->pieces_log < tile) ++p->pieces_log;
    return true;
}

}  // namespace

TOVL_API int tovl_page_plan(tovl_handle h, const tovl_page_plan_args* args, void* stream)
{
    if (!h || !args) return TOVL_ERR_INVALID;
    const auto [length, add, table, ring, state, length_out, state_out, slots, positions, starts, ldt, B, width, pages, page, cap] = *args;
    if (B < 0 || width < 1 || pages < 1 || page < 1 || cap < 0) return TOVL_ERR_INVALID;
    if (B > kMaxRequests || cap > kMaxNewTokens || static_cast<long long>(pages) * page > INT_MAX) return TOVL_ERR_UNSUPPORTED;
    if (B == 0) return TOVL_OK;
    if (!length || !add || !table || !ring || !state || !length_out || !state_out || !starts || (cap && (!slots || !positions)) ||
        ldt < width)
        return TOVL_ERR_INVALID;
    const void* all[] = {length, add, table, ring, state, length_out, state_out, slots, positions, starts};
    for (const void* p : all)
        if (!aligned(p, 4)) return TOVL_ERR_INVALID;
    PagePlanParams p = {};
    p.length = length;
    p.add = add;
    p.table = table;
    p.ring = ring;
    p.state = state;
    p.length_out = length_out;
    p.state_out = state_out;
    p.slots = slots;
    p.positions = positions;
    p.starts = starts;
    p.ldt = ldt;
    p.B = B;
    p.width = width;
    p.pages = pages;
    p.page = page;
    p.cap = cap;
    p.page_shift = shift_of(page);
    p.in_place = length_out == length || state_out == state;
    p.counter = h->sync_words + kPagePlanWord;
    p.ctrl = h->ctrl;
    DeviceGuard g(h->device);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return run(h, s, "page plan launch", [&](bool pdl) { return launch_page_plan(p, h->num_sms, s, pdl); });
}

TOVL_API int tovl_rope_append(tovl_handle h, const tovl_rope_append_args* args, void* stream)
{
    if (!h || !args) return TOVL_ERR_INVALID;
    const auto [q, k, v, q_out, positions, slots, cos_sin, cache, ldq, ldk, ldv, ldqo, T, Hq, max_pos, rot, interleaved] = *args;
    RopeParams p = {};
    const int rc = check_cache(cache, &p.cache);
    if (rc != TOVL_OK) return rc;
    const int D = p.cache.dim;
    if (T < 0 || Hq < 1 || rot < 0 || rot > D || (rot && (!cos_sin || max_pos < 1))) return TOVL_ERR_INVALID;
    if (rot % 16 || Hq > kMaxQueryHeads) return TOVL_ERR_UNSUPPORTED;
    if (T == 0) return TOVL_OK;
    if (!positions || !slots || !aligned(positions, 4) || !aligned(slots, 4) || (rot && !aligned16(cos_sin))) return TOVL_ERR_INVALID;
    const long long wide_q = static_cast<long long>(Hq) * D, wide_k = static_cast<long long>(p.cache.heads) * D;
    if (!valid_rows(q, ldq, wide_q) || !valid_rows(k, ldk, wide_k) || !valid_rows(v, ldv, wide_k) || !valid_rows(q_out, ldqo, wide_q))
        return TOVL_ERR_INVALID;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.positions = positions;
    p.slots = slots;
    p.cos_sin = cos_sin;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.ldqo = ldqo;
    p.T = T;
    p.Hq = Hq;
    p.rot = rot;
    p.max_pos = max_pos;
    p.interleaved = interleaved != 0;
    const bool e4m3 = cache->type == TOVL_E4M3;
    p.ctrl = h->ctrl;
    DeviceGuard g(h->device);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return run(h, s, "rotary embedding launch",
               [&](bool pdl) { return launch_rope_append(p, e4m3, h->num_sms, s, pdl); });
}

TOVL_API long long tovl_attn_decode_workspace(tovl_handle h, int Hq, int heads, int dim)
{
    if (!h || heads < 1 || Hq < 1 || Hq % heads || Hq > kMaxQueryHeads || dim < 1 || dim > kMaxHeadDim || dim % 8) return -1;
    return attn_decode_workspace(heads, Hq / heads, dim, h->num_sms);
}

TOVL_API int tovl_attn_decode(tovl_handle h, const tovl_attn_decode_args* args, void* stream)
{
    if (!h || !args) return TOVL_ERR_INVALID;
    const auto [q, out, lse, table, length, cache, workspace, ldq, ldo, ldt, workspace_bytes, B, Hq, width, window, scale] = *args;
    AttnParams p;
    std::memset(&p, 0, sizeof p);
    const int rc = check_cache(cache, &p.cache);
    if (rc != TOVL_OK) return rc;
    if (B < 0 || Hq < 1 || Hq % p.cache.heads || width < 1 || window < 0) return TOVL_ERR_INVALID;
    if (Hq > kMaxQueryHeads || B > kMaxDecodeBatch || h->num_sms > kMaxGrid) return TOVL_ERR_UNSUPPORTED;
    if (B == 0) return TOVL_OK;
    const long long wide = static_cast<long long>(Hq) * p.cache.dim;
    if (!valid_rows(q, ldq, wide) || !valid_rows(out, ldo, wide) || !table || !length || ldt < width || !aligned(table, 4) ||
        !aligned(length, 4) || !aligned(lse, 4) || !workspace || !aligned(workspace, 256) ||
        workspace_bytes < tovl_attn_decode_workspace(h, Hq, p.cache.heads, p.cache.dim))
        return TOVL_ERR_INVALID;
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.table = table;
    p.length = length;
    p.ldq = ldq;
    p.ldo = ldo;
    p.ldt = ldt;
    p.B = B;
    p.Hq = Hq;
    p.group = Hq / p.cache.heads;
    const long long held = static_cast<long long>(width) * p.cache.page;
    p.most_tokens = held < INT_MAX - 63 ? static_cast<int>(held) : INT_MAX - 63;
    p.window = window;
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.part = static_cast<float*>(workspace);
    p.counter = h->sync_words + kAttnWord;
    p.timeout_ns = 4 * h->timeout_ns + 100000000LL;
    p.ctrl = h->ctrl;
    DeviceGuard g(h->device);
    const bool e4m3 = cache->type == TOVL_E4M3;
    const AttnShape shape = attn_decode_shape(p.cache.dim, e4m3, p.group, false);
    const int row = p.cache.dim * (e4m3 ? 1 : 2), heads = p.cache.heads;
    const bool adjacent = heads > 1 && p.cache.head_stride == row && (p.cache.page == 1 || p.cache.slot_stride >= heads * row);
    int together = adjacent && p.group <= shape.heads ? attn_decode_together(shape, heads, p.cache.dim, e4m3) : 1;
    p.boxed = map_cache(h, &p, e4m3, shape, together);
    p.pair = p.boxed && attn_decode_pairs(p.cache.dim, e4m3, p.group);
    if (p.pair) together = 2;
    for (int n = together; n > 1; n /= 2) ++p.together_log;
    const AttnShape taken = p.pair ? attn_decode_shape(p.cache.dim, e4m3, p.group, true) : shape;
    const int groups = heads * ((p.group + taken.heads - 1) / taken.heads) / together, turns = taken.warps / together;
    p.by_page = FastDiv(p.cache.page);
    p.by_groups = FastDiv(groups);
    p.by_turns = FastDiv(turns);
    p.most_tiles = (INT_MAX - 1) / groups;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return run(h, s, "attention launch",
               [&](bool pdl) { return launch_attn_decode(p, e4m3, h->num_sms, s, pdl); });
}
