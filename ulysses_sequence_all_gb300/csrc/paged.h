// paged.h -- argument blocks of the kernels of the paged key-value cache, shared by api.cu,
// cache_append.cu and attention_paged.cu.
//
// A rank's keys (and values) lie in a pool of pages, (pages, page, m_r, d): the head-side tensor of a
// plan whose batch is the pages and whose sequence is a page. Key j of batch element bb is row
// j % page of page table[bb][j / page].
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "plan.h"

namespace uly {

constexpr int kPagedTile = 16;           // keys that a warp takes at a time
constexpr int kPagedWarps = 4;
constexpr int kPagedBlock = kPagedTile * kPagedWarps;
// Query rows a key head (group * tokens) up to which attention_paged.cu runs, above them the tensor cores'
// long layout. Over pages, paged : long in us, 8, 16, 32 rows: 8 caches of 3,000-9,000 tokens, 8 key heads 46 : 72,
// 49 : 73, 51 : 74; 16 of 12,000-32,000, 4 key heads 128 : 195, 131 : 196, 133 : 197; 256 of 100-2,000, 8 key heads
// 180 : 357, 200 : 358, 230 : 359; 32 windows of 4,096, 20 rows 106 : 123. (With 64 rows, 16 for each of the four
// warps, it took 67 : 71, 203 : 193, 381 : 353, 176 : 124: no such form is kept.)
constexpr int kPagedFewRows = 32;
// Over contiguous keys with a window of 4,096, 8 key heads, 4, 16, 32 rows: 4 caches 20.6 : 25.7, 24.8 : 25.5,
// 27.8 : 26.7; 32 caches 91 : 105, 99 : 105, 104.6 : 105.4.
constexpr int kWindowFewRows = 16;

struct AppendArgs {
    const uint8_t* src[2][kMaxW];  // new keys, values: (b, tokens, m_r, d)
    uint8_t* dst[2][kMaxW];        // pools: (pages, page, m_r, d)
    uint32_t words[kMaxW];         // 16-byte words of a token, m_r * d * e / 16
    const int32_t *table, *starts, *counts;  // counts: null (all tokens)
    int64_t b, tokens, table_pages;
    int64_t pages, page;
    int32_t W;
};

// A sequence (a batch element's key head) that several shares of the work have parts of: share `cta` its
// beginning, the next parts - 1 the rest.
struct PagedShared {
    int32_t parts;  // 0: none
    int32_t cta, bb, head;
};

struct PagedArgs {
    CUtensorMap kmap[kMaxW], vmap[kMaxW];  // boxes of `box` rows of a page, one head
    const uint8_t* q[kMaxW];
    uint8_t* o[kMaxW];
    float* lse[kMaxW];
    int32_t n[kMaxW], m_begin[kMaxW + 1];  // query heads; prefix of key heads over the ranks
    const int32_t* table;    // (b, table_pages); null: batch element bb's only page is bb
    const int32_t* kv_lens;  // (b) or null: `room`
    const int32_t* q_start;  // (b) or null: from_end: the keys' count less Sq, else zeros
    int64_t Sq, table_pages;
    int32_t W, b, d, group, f16;
    int32_t pages, page, box, from_end;
    int32_t room;            // keys that a batch element's pages can hold
    int32_t sinks;
    int64_t window;          // beyond every position where there is none
    int32_t rows;    // query rows of the kernel (8, 16, 32), of which the call's are the first
    int32_t parts;   // shares of all the work, one CTA at a time works on one
    int32_t end;     // blocks that a sequence's end counts for in them
    int32_t by_sequence, notes;  // `shared` has an entry for each sequence, or for each share
    float scale;
    uint32_t wait_us;
    float* part_o;         // [2 parts][rows][d] normalised partial outputs
    float* part_lse;       // [2 parts][rows]
    PagedShared* shared;   // [notes], at most parts
};

cudaError_t cache_append_launch(const AppendArgs& a, cudaStream_t stream, int64_t cap, int sm_count);
// Rows and shares from the shape and the device alone: a CTA cap changes no bit.
void attn_paged_split(PagedArgs* a, int sm_count);
cudaError_t attn_paged_launch(PagedArgs& a, const void* const* k, const void* const* v,
                              cudaStream_t stream, int device, int64_t cap);
cudaError_t cache_append_status(unsigned* status, bool clear);
cudaError_t attn_paged_status(unsigned* status, bool clear);

}  // namespace uly
