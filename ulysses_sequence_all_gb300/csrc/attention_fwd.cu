// attention_fwd.cu -- host side of the attention forward (see attention_fwd.cuh): units and parts, tensor
// maps, and the launches without a window. attention_fwd_window.cu and attention_fwd_pages.cu hold the others,
// so that they compile side by side.
#include "attention_fwd.cuh"

namespace uly {

int64_t attn_order_group(int64_t heads, int64_t bytes)
{
    int64_t g = (int64_t(64) << 20) / (bytes > 0 ? bytes : 1);
    if (g > 256) g = 256;
    if (g > heads) g = heads;
    return g < 1 ? 1 : g;
}

bool encode_sink_maps(const AttnShape& s, int r, const void* k, const void* v, CUtensorMap* k_sink,
                      CUtensorMap* v_sink, CUtensorMap* k_rest, CUtensorMap* v_rest)
{
    if (!s.window || s.sink_rows == 0 || s.sink_rows >= kAttnRows) return true;
    const int64_t rest = kAttnRows - s.sink_rows;
    return encode_head_map(k_sink, k, s.f16, s.d, s.m[r], s.Skv, s.b, 1, s.sink_rows) &&
           encode_head_map(v_sink, v, s.f16, s.d, s.m[r], s.Skv, s.b, 1, s.sink_rows) &&
           encode_head_map(k_rest, k, s.f16, s.d, s.m[r], s.Skv, s.b, 1, rest) &&
           encode_head_map(v_rest, v, s.f16, s.d, s.m[r], s.Skv, s.b, 1, rest);
}

// Row tiles, units and parts of the keys. Where one tile holds all rows, a CTA's two tiles take a
// part each. The keys are split further while a part keeps some blocks (a part costs its start, an
// fp32 output and a share of the join).
// Key blocks of a unit at most.
static int64_t af_most_blocks(const AttnShape& s, int64_t pair)
{
    const int64_t all = (s.Skv + kAttnRows - 1) / kAttnRows;
    if (!s.window) return all;
    // (a window of w keys over `pair` tokens; the first tokens)
    const int64_t near = s.window >= s.Skv ? s.Skv : s.window + pair - 1;
    const int64_t some = (near + s.sink_rows + kAttnRows - 1) / kAttnRows;
    return some < all ? some : all;
}

void attn_fwd_split(AttnFwdArgs* a, int sm_count)
{
    const AttnShape& s = a->s;
    a->tile_tokens = kAttnRows / s.group;
    const int64_t pair = 2 * int64_t(a->tile_tokens);
    const int64_t blocks = af_most_blocks(s, pair);
    a->paired = !s.window && s.Sq <= a->tile_tokens && blocks > 1;
    if (a->paired) a->tile_tokens = int32_t(s.Sq);
    a->order.heads = s.head_begin[s.W];
    a->order.blocks = a->paired ? 1 : (s.Sq + pair - 1) / pair;
    // keys and values (with a window, those of a unit)
    a->order.group =
        attn_order_group(a->order.heads, (s.window ? blocks * kAttnRows : s.Skv) * s.d * 4);
    const int64_t base = a->order.heads * a->order.blocks;
    // One wave of the SMs (finer parts of a ragged batch, evened out by stealing, measured no faster:
    // 16 caches of 4 key heads 134 us with 2 units a head, 134 with 7, 136 with 9, 154 with 19; no other
    // number of heads was measured, and between half as many units as SMs and all of them, where n is
    // 1, the rest of the SMs have none), of a block a tile at least where rows are few (latency), of
    // four blocks where a part's output is a whole tile.
    int64_t n = base > 0 ? sm_count / base : 1;
    const int64_t most = blocks / (a->paired ? 2 : 4);
    if (n > most) n = most;
    const int64_t cap = kAfMaxParts / (a->paired ? 2 : 1);
    if (n > cap) n = cap;
    if (n < 1) n = 1;
    a->splits = int32_t(n);
    a->parts = a->paired ? 2 * a->splits : a->splits;
    a->units = base * a->splits;
}

// The keys are split where that leaves SMs idle, whatever the tables have room for (a part without keys
// says so): one wave of the SMs. None : half a wave : one : two : four, in us, 64 rows a key head: 16 caches
// of 12,000-32,000 tokens, 4 key heads 348 : 348 : 200 : 207 : 189, 8 of 30,000, 8 key heads 380 : 380 : 206 :
// 216 : 214, one of them 377 : 61 : 48 : 51 : 66, 8 of 3,000-9,000 121 : 121 : 76 : 82 : 84 (256 rows 135 : 135 : 94 : 106 :
// 122), 4 of 700 18.6 : 17.6 : 18.6 : 22 : 28; 512 tokens on 30,000, 32 heads over 8 369 : 370 : 213 : 228 : 236.
void attn_fwd_split_pages(AttnFwdArgs* a, int sm_count)
{
    const AttnShape& s = a->s;
    a->tile_tokens = kAttnRows / s.group;
    a->paired = 0;
    const int64_t pair = 2 * int64_t(a->tile_tokens), heads = s.head_begin[s.W];
    a->order = {heads, (s.Sq + pair - 1) / pair, attn_order_group(heads, s.Skv * s.d * 4)};
    const int64_t base = heads * a->order.blocks;
    int64_t n = base > 0 ? sm_count / base : 1;
    n = n > kAfMaxParts ? kAfMaxParts : n < 1 ? 1 : n;
    a->splits = a->parts = int32_t(n);
    a->units = base * n;
}

static cudaError_t af_launch(const AttnFwdArgs& a, cudaStream_t stream, int device, int64_t cap, int sm_count)
{
    if (a.pages.table) return attn_fwd_pages_launch(a, stream, device, cap, sm_count);
    if (a.s.window) return attn_fwd_window_launch(a, stream, device, cap, sm_count);
    if (a.paired)
        return a.tile_tokens * a.s.group <= kAfTokenRows
                   ? af_launch_types<kAfToken, false, false>(a, stream, device, cap, sm_count)
                   : af_launch_types<kAfPaired, false, false>(a, stream, device, cap, sm_count);
    if (a.s.d > 64) {  // (d <= 64 has room for both)
        const int64_t blocks = (a.s.Skv + kAttnRows - 1) / kAttnRows;
        const bool padded = a.s.kv_lens && a.s.b == 1;
        if (blocks <= int64_t(padded ? kAfShortBlocksPadded : kAfShortBlocks) * a.splits)
            return a.s.f16 ? af_launch_mode<128, true, kAfShort, false, false>(a, stream, device, cap, sm_count)
                           : af_launch_mode<128, false, kAfShort, false, false>(a, stream, device, cap, sm_count);
    }
    return af_launch_types<kAfLong, false, false>(a, stream, device, cap, sm_count);
}

// One launch over all ranks (and the join). The shape, outputs, parts and their buffers are set in
// `a`.
cudaError_t attn_fwd_launch(AttnFwdArgs& a, const void* const* q, const void* const* k,
                            const void* const* v, cudaStream_t stream, int device, int64_t cap,
                            int sm_count)
{
    const AttnShape& s = a.s;
    if (a.units == 0) return cudaSuccess;
    for (int r = 0; r < s.W; ++r) {
        if (s.n[r] == 0) continue;
        const AttnPages& p = a.pages;
        const int64_t rows = p.table ? p.page : s.Skv, b = p.table ? p.pages : s.b;
        const int64_t box = p.table ? p.box : kAttnRows;
        if (!encode_head_map(&a.qmap[r], q[r], s.f16, s.d, s.n[r], s.Sq, s.b, s.group, a.tile_tokens) ||
            !encode_head_map(&a.kmap[r], k[r], s.f16, s.d, s.m[r], rows, b, 1, box) ||
            !encode_head_map(&a.vmap[r], v[r], s.f16, s.d, s.m[r], rows, b, 1, box))
            return cudaErrorInvalidValue;
        if (p.table) continue;
        if (!encode_sink_maps(s, r, k[r], v[r], &a.kmap_sink[r], &a.vmap_sink[r], &a.kmap_rest[r],
                              &a.vmap_rest[r]))
            return cudaErrorInvalidValue;
    }
    return af_launch(a, stream, device, cap, sm_count);
}

cudaError_t attn_fwd_status(unsigned* status, bool clear)
{
    unsigned w = 0, p = 0;
    cudaError_t e = af_status(status, clear);
    if (e == cudaSuccess) e = attn_fwd_window_status(&w, clear);
    if (e == cudaSuccess) e = attn_fwd_pages_status(&p, clear);
    *status |= w | p;
    return e;
}

}  // namespace uly
