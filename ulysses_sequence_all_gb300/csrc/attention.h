// attention.h -- argument blocks of the attention kernels, shared by api.cu and attention_*.cu.
//
// All W ranks' heads run in one launch. Queries (b, Sq, n_r, d) and keys, values (b, Skv, m_r, d)
// are the head-side tensors that mode 0 writes; `group` = n_r / m_r query heads share a key head.
// A row tile is 128 rows of one (rank, batch element, key head): `tile_tokens` = 128 / group tokens
// with their `group` heads each, row = token * group + head, so that shared heads read their keys
// once. Rows past tile_tokens * group are computed on whatever lies there and never stored.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "plan.h"
#ifdef __CUDACC__
#include "tcgen05.cuh"
#endif

namespace uly {

constexpr int kAttnMaxD = 128;
constexpr int kAttnMaxGroup = 64;  // query heads that share a key head
constexpr int kAttnRows = 128;     // rows of a query tile, and keys of a block
constexpr int kAttnPBits = 14;     // fp16 probabilities of the backward are held times 2^this

// What every attention kernel needs to know of the call.
struct AttnShape {
    int64_t Sq, Skv;
    int32_t W, b, d, f16;
    int32_t group;
    int32_t n[kMaxW], m[kMaxW];      // query and key heads of each rank
    int32_t head_begin[kMaxW + 1];   // prefix of b * m_r over the ranks: (rank, batch, key head)
    int64_t row_begin[kMaxW + 1];    // prefix of b * n_r * Sq: rows of the log-sum-exp arrays
    const int32_t* kv_lens;          // (b) or null: keys of each batch element, clamped to [0, Skv]
    const int32_t* q_start;          // (b) or null (zeros): position of the first query, causal only
    int32_t causal;
    // Whether a block can hold keys that no row sees next to ones that rows do: what they hold is not
    // used, whatever it is (key counts; causal, keys past the last row's position).
    int32_t ragged;
    uint32_t wait_us;  // limit of a wait in which nothing moves (CtaLife)
    float scale;
    // Causal with a window (0: none): the query at position p sees j <= p with j > p - window or j < sinks.
    int32_t sinks;
    int32_t sink_rows;  // rows that they take in a unit's blocks: see AttnBlocks
    int64_t window;
    int32_t align;      // a unit's window begins at a multiple of this (1; pages: rows of a copy)
    int32_t from_end;   // without q_start the queries are the last Sq tokens
};
// Up to here first tokens share a block with keys of the window (a copy of 8 k rows in front of theirs);
// more of them have blocks of their own.
constexpr int kAttnSharedSinks = 64;

#ifdef __CUDACC__
// Keys of batch element bb that any row sees, and the position of its first query (beyond every key
// when the mask is not causal).
__device__ __forceinline__ void attn_limits(const AttnShape& s, int bb, int64_t* len, int64_t* pos0)
{
    *len = s.kv_lens ? min(s.Skv, int64_t(max(0, s.kv_lens[bb]))) : s.Skv;
    *pos0 = s.Skv;
    if (s.causal) {
        *pos0 = s.q_start ? int64_t(s.q_start[bb]) : s.from_end ? *len - s.Sq : 0;
        *len = min(*len, max(int64_t(0), *pos0 + s.Sq));
    }
}
#endif

// The key blocks that a unit walks are rows 128 j .. 128 j + 127 of its list of keys: 0, 1, ...; with a
// window the first tokens (rows below `pad`, of which those from `sinks` on are masked), then the keys
// from `begin` on, the first in the window of the unit's first row. So that a list has no row before its
// window, blocks begin at any key.
#ifdef __CUDACC__
template <bool WIN>
struct AttnBlocks {
};
template <>
struct AttnBlocks<true> {
    int pad, begin;
    // `first`: the first key in the first row's window, at most `end`, that of the keys anyone sees
    __device__ __forceinline__ void set(const AttnShape& s, int64_t first, int64_t end)
    {
        if (first < end && s.align > 1) first -= first % s.align;
        const bool apart = first > s.sink_rows;
        pad = apart ? s.sink_rows : 0;
        begin = apart ? int(first) : 0;
    }
    // Rows that hold the keys below `end` that anyone may see.
    __device__ __forceinline__ int rows(const AttnShape& s, int64_t end) const
    {
        return end > begin ? int(end - begin) + pad : pad ? int(max(int64_t(0), min(int64_t(s.sinks), end))) : 0;
    }
    __device__ __forceinline__ int key(int row) const { return row < pad ? row : row - pad + begin; }
    // The rows of block j that hold what no row of the batch element sees between the first tokens and its
    // first window, or first tokens that are none: x .. y - 1 (none where y <= x).
    __device__ __forceinline__ int2 between(const AttnShape& s, int64_t pos0, int j) const
    {
        const int64_t to = pad + max(int64_t(0), pos0 + 1 - s.window - begin), row0 = int64_t(j) * kAttnRows;
        return make_int2(int(max(int64_t(0), min(int64_t(kAttnRows), s.sinks - row0))),
                         int(max(int64_t(0), min(int64_t(kAttnRows), to - row0))));
    }
};

// Copies key block j (of a list, with a window) of a head: the `halves` tiles of 64 columns, kHalf apart.
template <bool WIN, int HALF>
__device__ __forceinline__ void attn_load_keys(uint8_t* to, int halves, const CUtensorMap* map,
                                               const CUtensorMap* sink_map, const CUtensorMap* rest_map,
                                               const AttnBlocks<WIN>& list, int head, int j, int bb,
                                               uint64_t* bar)
{
    if constexpr (WIN) {
        if (j == 0 && list.pad > 0 && list.pad < kAttnRows) {
            for (int h = 0; h < halves; ++h) {
                tensor_g2s_4d(to + h * HALF, sink_map, 64 * h, head, 0, bb, bar);
                tensor_g2s_4d(to + h * HALF + list.pad * 128, rest_map, 64 * h, head, list.begin, bb, bar);
            }
            return;
        }
        for (int h = 0; h < halves; ++h)
            tensor_g2s_4d(to + h * HALF, map, 64 * h, head, list.key(j * kAttnRows), bb, bar);
    } else {
        for (int h = 0; h < halves; ++h)
            tensor_g2s_4d(to + h * HALF, map, 64 * h, head, j * kAttnRows, bb, bar);
    }
}
#endif

// Order of the units of a kernel: groups of `group` heads, in a group by block (the longest first
// when they differ), then by head. A group's shared operands fit the L2 cache.
struct AttnOrder {
    int64_t heads, blocks, group;
};

#ifdef __CUDACC__
__device__ __forceinline__ void attn_order(const AttnOrder& o, int64_t u, int64_t* head,
                                           int64_t* block)
{
    const int64_t per = o.group * o.blocks;
    const int64_t g = per > u ? 0 : div_fast(u, per);
    const int64_t at = u - g * per, heads = min(o.group, o.heads - g * o.group);
    *block = heads == 1 ? at : div_fast(at, heads);
    *head = g * o.group + (at - *block * heads);
}

// A CTA's units, asked for by one whole warp, the one that watches (CtaLife). A grid of one CTA per unit (gridDim.x == units): its
// own, then those of CTAs that have not started, which it takes their place of as it gets there, so
// that long and short units even out. A smaller grid (a CTA cap): every gridDim.x-th unit, back and
// forth, which evens out units whose length falls along the order.
struct AttnUnitSource {
    int64_t units;
    void* answer;     // 16 bytes of shared memory
    uint64_t* bar;    // counts the answer; initialised for one arrival
    volatile CtaLife* life;
    int64_t wave = 0;
    uint32_t phase = 0;
    bool over = false;
    __device__ __forceinline__ int64_t next()  // -1: no more
    {
        const int64_t grid = gridDim.x;
        if (grid < units) {
            while (wave * grid < units) {
                const int64_t c = (wave & 1) ? grid - 1 - blockIdx.x : blockIdx.x;
                const int64_t u = wave++ * grid + c;
                if (u < units) return u;
            }
            return -1;
        }
        if (wave++ == 0) return blockIdx.x;
        if (over) return -1;
        if ((threadIdx.x & 31) == 0) {
            fence_proxy_async_shared();
            mbar_arrive_expect_tx(bar, 16);
            steal_cta(answer, bar);
        }
        __syncwarp();
        const bool ok = __all_sync(0xffffffffu, wait_watching(bar, phase, life));
        // (an answer on its way lands before this CTA's shared memory may be another's)
        if (!ok && !mbar_wait_bounded(bar, phase)) life->stuck = 1;
        phase ^= 1u;
        const int64_t u = ok ? stolen_cta(answer) : -1;
        __syncwarp();
        over = u < 0;
        return u;
    }
};
#endif

// Keys and values in pages (see paged.h): key j of batch element bb is row j % page of page
// table[bb][j / page]; a copy takes `box` rows of one.
struct AttnPages {
    const int32_t* table;
    int64_t table_pages;
    int32_t pages, page, box;
};

struct AttnFwdArgs {
    AttnShape s;
    AttnPages pages;
    CUtensorMap qmap[kMaxW], kmap[kMaxW], vmap[kMaxW];
    CUtensorMap kmap_sink[kMaxW], vmap_sink[kMaxW];  // with a window: boxes of sink_rows, and of the rest
    CUtensorMap kmap_rest[kMaxW], vmap_rest[kMaxW];  // of a block
    uint8_t* o[kMaxW];
    float* lse[kMaxW];  // (b, n_r, Sq)
    int32_t tile_tokens;
    AttnOrder order;    // (rank, batch, key head) x pairs of row tiles along the tokens
    int64_t units;      // the same, x splits
    int32_t splits;     // units along the keys
    int32_t paired;     // a unit's two tiles are the same rows, each with its own part of the keys
    int32_t parts;      // parts of the keys (splits, or twice as many when paired)
    float* part_o;      // [parts][rows][d] normalised partial outputs, parts > 1, joined by a
    float* part_lse;    // [parts][rows]    second kernel
};

struct AttnBwdArgs {
    AttnShape s;
    CUtensorMap qmap[kMaxW], gmap[kMaxW];  // boxes of a row tile: q, dO
    CUtensorMap kmap[kMaxW], vmap[kMaxW];  // boxes of a key block
    CUtensorMap kmap_sink[kMaxW], vmap_sink[kMaxW];  // dQ with a window: as the forward's
    CUtensorMap kmap_rest[kMaxW], vmap_rest[kMaxW];
    const uint8_t* o[kMaxW];
    const uint8_t* go[kMaxW];
    const uint8_t* v[kMaxW];
    const float* lse[kMaxW];
    uint8_t* dq[kMaxW];
    uint8_t* dk[kMaxW];
    uint8_t* dv[kMaxW];
    int32_t tile_tokens;
    int64_t q_tiles;              // row tiles along the tokens
    AttnOrder q_order, kv_order;  // (rank, batch, key head) x row tiles, x key blocks
    // [(rank, batch, key head)][q_tiles][2][128]: lse in powers of two, delta; fp16 [3][128], the lse
    // less kAttnPBits, and |dO|
    float* stats;
    float2* row_bounds;  // fp16: [(rank, batch, key head)][q_tiles][2]: largest |dO|, |delta| of half a tile
    float* key_norms;    // fp16: [(rank, batch, key head)][key blocks]: largest |v|
    // With a window: dK, dV's units. A block of first tokens is seen by every later row; its row tiles are
    // cut into `chunks` units of chunk_tiles each, whose sums for the first tokens go to `part`,
    // [(rank, batch, key head)][sink_keys][chunks][2][d] fp32, and are added in order by a last kernel.
    AttnOrder kv_units;  // (rank, batch, key head) x (blocks, those of the first tokens chunks times)
    int32_t sink_keys, sink_blocks, chunks;
    int64_t chunk_tiles;
    float* part;
    uint32_t* ready;  // 0 from the statistics kernel, 1 from dK, dV's once it has seen the statistics
};

// Host side.
constexpr int64_t kAttnMostCtas = 0x7FFFFFFF;  // of a grid, and the cap of a plan without one
// CTAs of a launch of `units`: one each, to be taken over by those that are done (AttnUnitSource);
// where the plan's cap or a grid holds fewer, as many as run at a time.
inline unsigned attn_ctas(int64_t units, int64_t cap, int sm_count)
{
    return unsigned(units <= cap ? units : cap < sm_count ? cap : sm_count);
}
// A launch that may start before the kernel in front of it has finished (see let_next_start); the
// kernel itself waits where it needs that (wait_for_previous). early = false: an ordinary launch.
template <class Args>
inline cudaError_t attn_launch_early(void (*kernel)(Args), unsigned grid, unsigned block, int smem,
                                     cudaStream_t stream, const Args& a, bool early = true)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Heads in a group: as many as hold `bytes` each within about half of the L2 cache. The heads of a
// token lie next to one another, so the CTAs at work then read whole stretches of memory; with
// longer operands a head at a time keeps those in the cache.
int64_t attn_order_group(int64_t heads, int64_t bytes);
// Tiles, units and parts of the keys from the shape and the device alone: a CTA cap changes no bit.
void attn_fwd_split(AttnFwdArgs* a, int sm_count);
// The same over pages, whatever their tables have room for.
void attn_fwd_split_pages(AttnFwdArgs* a, int sm_count);
// Maps of a block that first tokens share with keys of the window (where there is one).
bool encode_sink_maps(const AttnShape& s, int r, const void* k, const void* v, CUtensorMap* k_sink,
                      CUtensorMap* v_sink, CUtensorMap* k_rest, CUtensorMap* v_rest);
// The units of dK, dV with a window, from the shape and the device alone.
void attn_bwd_split(AttnBwdArgs* a, int sm_count);
// `cap`: CTAs of a launch at most; under one (below kAttnMostCtas) no kernel starts beside another.
cudaError_t attn_fwd_launch(AttnFwdArgs& a, const void* const* q, const void* const* k,
                            const void* const* v, cudaStream_t stream, int device, int64_t cap,
                            int sm_count);
cudaError_t attn_fwd_status(unsigned* status, bool clear);
cudaError_t attn_fwd_window_launch(const AttnFwdArgs& a, cudaStream_t stream, int device, int64_t cap,
                                   int sm_count);
cudaError_t attn_fwd_window_status(unsigned* status, bool clear);
cudaError_t attn_fwd_pages_launch(const AttnFwdArgs& a, cudaStream_t stream, int device, int64_t cap,
                                  int sm_count);
cudaError_t attn_fwd_pages_status(unsigned* status, bool clear);
cudaError_t attn_bwd_launch(AttnBwdArgs& a, const void* const* q, const void* const* k,
                            const void* const* v, cudaStream_t stream, int device, int64_t cap,
                            int sm_count);
cudaError_t attn_bwd_status(unsigned* status, bool clear);

}  // namespace uly
