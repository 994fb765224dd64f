// paged.cuh -- parameter blocks and launchers of the paged attention step:
// pages for new tokens, rotary embedding with the cache writes, attention of
// one new token per request.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include "ctrl.cuh"
#include "ops.cuh"

namespace tovl {

constexpr int kMaxRequests = 4096;     // of one page_plan call
constexpr int kMaxHeadDim = 256;

// Division by a number that the host knows, of x < 2^31.
struct FastDiv {
    unsigned long long m;
    int s;
    FastDiv() = default;
    explicit FastDiv(unsigned d) : s(31)
    {
        while (1ull << (s - 31) < d) ++s;
        m = ((1ull << s) + d - 1) / d;      // at most 2^32; m d - 2^s < d <= 2^(s - 31)
    }
    __host__ __device__ int div(unsigned x) const { return static_cast<int>(x * m >> s); }
};

// tovl_kv_cache with strides in bytes.
struct KvCache {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;         // [pages][heads][page]; e4m3 only
    float* v_scale;
    long long page_stride, slot_stride, head_stride;
    int pages, page, heads, dim;
    int page_shift;         // log2(page), or -1
};

struct PagePlanParams {
    const int* length;      // [B]
    const int* add;         // [B]
    int* table;             // [B][width], rows ldt apart
    int* ring;              // [pages]
    const int* state;       // [4]
    int* length_out;
    int* state_out;
    int* slots;             // [cap]
    int* positions;         // [cap]
    int* starts;            // [B + 1]
    long long ldt;
    int B, width, pages, page, cap;
    int page_shift;         // log2(page), or -1
    int in_place;           // length_out is length, or state_out state
    int* counter;           // handle-owned, zero between calls
    Ctrl ctrl;
};
cudaError_t prepare_page_plan();
cudaError_t launch_page_plan(const PagePlanParams& p, int num_sms, cudaStream_t stream, bool pdl);

struct RopeParams {
    const void* q;          // bf16 [T][Hq][D], rows ldq elements apart
    const void* k;          // bf16 [T][heads][D]
    const void* v;
    void* q_out;
    const int* positions;   // [T]
    const int* slots;       // [T]
    const float* cos_sin;   // [max_pos][rot]
    long long ldq, ldk, ldv, ldqo;
    int T, Hq, rot, max_pos, interleaved;
    KvCache cache;
    Ctrl ctrl;
};
cudaError_t launch_rope_append(const RopeParams& p, bool e4m3, int num_sms, cudaStream_t stream, bool pdl);

struct AttnParams {
    const void* q;          // bf16 [B][Hq][D], rows ldq elements apart
    void* out;              // rows ldo apart
    float* lse;             // [B][Hq]; null = not wanted
    const int* table;       // [B][width], rows ldt apart
    const int* length;      // [B]
    long long ldq, ldo, ldt;
    int B, Hq, group, window;
    int most_tokens;        // of a request
    float scale_log2;       // scale * log2(e)
    KvCache cache;
    // boxed: pages are copied in boxes of 64 or 128 bytes of columns x rows of one
    // head; dimensions of the maps: columns, heads, slots (slots_first: slots,
    // heads), pages
    CUtensorMap k_map, v_map;
    int boxed, slots_first;
    int pieces_log;         // log2 of the boxes that make the rows of a tile
    float* part;            // workspace
    int together_log;       // log2 of the heads that neighbouring warps take side by side
    int pair;               // attn_decode_pairs: they are two blocks of one key head
    int* counter;           // [24 * kMaxGrid], handle-owned, zero between calls
    FastDiv by_page, by_groups, by_turns;      // turns: warps that take a segment's tiles in turn
    unsigned most_tiles;    // of a head: below 2^31 - 1 in all, where the kernel's sums stop
    long long timeout_ns;
    Ctrl ctrl;
};
// Rows of a tile, bytes of a box's columns, warps of a CTA, query heads that a
// warp takes, floats of a part.
struct AttnShape {
    int rows, box_bytes, warps, heads, part;
};
AttnShape attn_decode_shape(int dim, bool e4m3, int group, bool pair);
// Key heads that neighbouring warps take side by side (1, 2, 4 or 8) where the
// heads of a slot are adjacent: so many that their rows are whole 128-byte lines.
// Read at other times, a line's halves come from memory twice.  Alone and side by
// side, us: 64 requests of 8192 tokens, 8 heads of 64, e4m3 197 and 139, bf16 198
// and 182; 64 of 4096, 8 heads of 80, bf16 186 and 138.
int attn_decode_together(const AttnShape& s, int heads, int dim, bool e4m3);
// bf16 heads of more than 128 columns with an even number of blocks of 8 query
// heads: two warps take two blocks from one ring, which leaves the shared memory
// for 12 warps (with rings of their own: 6).  32 requests up to 8192 tokens, 1 head
// of 256 for 16: 39 us, with rings of their own 41; with 16 heads a warp the sums do
// not fit the registers.
bool attn_decode_pairs(int dim, bool e4m3, int group);
long long attn_decode_workspace(int heads, int group, int dim, int num_sms);
cudaError_t prepare_attn_decode();
cudaError_t prepare_attn_decode_e4m3();
cudaError_t launch_attn_decode_e4m3(const AttnParams& p, int num_sms, cudaStream_t stream, bool pdl);
cudaError_t launch_attn_decode(const AttnParams& p, bool e4m3, int num_sms, cudaStream_t stream, bool pdl);

}  // namespace tovl
