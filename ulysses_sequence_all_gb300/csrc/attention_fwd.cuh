// attention_fwd.cuh -- attention of every rank's heads over the whole sequence, between the two
// relayouts (fast-ulysses 0.2.1, README, "Quick start": the attention of a sequence-parallel block
// runs on the head shards that mode 0 delivers).
//
// Per query row i of a head, over the keys j that it sees (j below the batch element's key count
// and, causal, j <= position of i): o_i = sum_j exp(s_ij - m_i) v_j / l_i, s_ij = scale q_i . k_j,
// m_i = max_j s_ij, l_i = sum_j exp(s_ij - m_i), and lse_i = m_i + log l_i. A row that sees no key
// gives zeros and lse = -infinity.
//
// One pass over the keys in blocks of 128 with the running maximum and sum: 4 d flops per (row,
// key) on the tensor cores, one exponential. With d = 128 it is bound by the products, those of S
// by reading both operands from shared memory (about 107 cycles each in place of 64); with few rows
// by reading the keys. Measured: 75,600 tokens x 8 heads of 128 in 13.7-13.8 ms, 1.69-1.70 PFLOP/s
// (0.86 of the measured cuBLAS rate); 2 x 4,095 causal tokens, 32 heads over 8, in 0.197 ms; one
// token each on 16 caches of 12,000-32,000 keys in 0.126 ms (0.81 of the copy peak).
//
// A CTA (one per SM, 384 threads) takes two tiles of 128 query rows that share their keys, unit
// after unit. Warp 11 works out the units ahead and leaves their records in shared memory. Warp 8
// loads (tensor maps, swizzled): query tiles into a few slots, so that the next unit's arrive
// during this one, and key and value blocks into a ring. One lane of warp 9 issues the products:
// S = Q K^T of one tile while the other tile's 128 threads turn their S into probabilities, so the
// tensor cores always have one tile's work; a unit's first scores follow the last unit's products
// without a gap. Warps 0-3 and 4-7 are the two tiles' softmax: tensor memory gives a thread a whole
// row, so maximum and sum need no exchange; they hold most of the registers. Warp 10 zeroes what a
// value block holds past the last key that any row of its batch element sees. Warp 11 also watches that
// the others get on (CtaLife).
// P goes back to tensor memory over its own S in 16 bits, rounded to nearest (unit-scale values
// in an fp32 sum: the output itself is rounded to the same type), and is the A operand of O += P V
// there, whose first half starts when half of P is written. O stays in tensor memory; it is
// rescaled only when a row's maximum has grown by more than 2^8 since its last scale (P then stays
// below 2^8, inside either type, fp16 times 2^7), by the softmax threads themselves: the block's S is complete
// only after the previous O product. They also write the finished rows, turned in the query tile's
// slot so that a store covers whole 128-byte lines.
//
// Sums: l in fp32, every term rounded to nearest; O in the tensor cores' fp32 accumulators, which cut off
// what lies below their last bit: O is too small by up to 2^-23 of itself for every 16 keys of a part
// (0.02 % at 25,000 keys, 0.05 % at 75,600; measured at 100,000: 0.035 %).
//
// With a window (WIN) the row at position p sees keys j <= p with j > p - window or j < sinks. A unit's blocks
// are those of its list of keys (AttnBlocks): the first tokens, then from its first row's window on, whatever
// key that is; blocks without an edge of any row's are not masked. Bound as above, each unit's start and end
// (about 4 us) weighing more the shorter its list is. Measured: 75,600 tokens x 8 heads of 128, window 10,800
// and 3,600 first tokens in 2.45-2.62 ms, 1.54-1.64 PFLOP/s; 2 x 4,095 tokens, 32 heads over 8, window 1,024
// and 4 first tokens in 0.117-0.133 ms, of whose cycles the tensor pipe is busy in 43 %.
// Over pages (PAGED) the loading warp's lanes copy a page's rows each, its place in the table looked up a block
// ahead; list rows that no row sees are copied from beyond the pool, which gives zeros. Measured: 8 caches of
// 30,000 tokens, 8 key heads, 64 rows each in 205 us (0.71 of the copy peak), pages of 32 tokens; pieces of prompts,
// 32 heads over 8 of 128, pages of 64: the last 2,048 of 8,000 tokens, 4 of them, in 640 us (1.46 PFLOP/s), of
// 30,000, 2 of them, in 1.42 ms (1.37); whole prompts, 2 x 4,095, in 223 us (1.23 PFLOP/s; contiguous keys 183 us).
//
// With few rows (one tile of them: single tokens) both tiles of a CTA are those rows, each over its
// own part of the keys; with too few units to fill the SMs the keys are split further. A part has
// its own normalised fp32 output and lse, and attn_join_kernel adds them weighted by
// exp(lse_part - lse).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "../../include/ulysses.h"
#include "attention.h"
#include "fused_row.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace uly {

static __device__ unsigned g_attn_fwd_status;

constexpr int kAfThreads = 384;
constexpr int kAfLoadWarp = 8, kAfMmaWarp = 9, kAfCleanWarp = 10, kAfUnitWarp = 11;
constexpr int kAfMaxUnitSlots = 4;
constexpr int kAfBarBytes = 1024;
constexpr int kAfMaxParts = 64;   // of the keys
// Key blocks of a unit up to which it counts as short; more of them for one batch element with a key
// count (a padded text), whose tensor has room that the count, which the host does not see, may leave
// unused. 75,600 queries x 40 heads of 128, short : long in us. No counts: 77 keys 377 : 426, 256
// 477 : 481, 384 616 : 561, 512 751 : 671. One element that holds all, 5/6, 2/3, 1/2, 1/3 of 384 keys:
// 606 : 588, 620 : 620, 622 : 619, 528 : 585, 405 : 456; of 512: 739 : 692, 743 : 725, 620 : 623,
// 490 : 526, 526 : 585 (so a full one loses 3 and 7 % by the rule, a third of one gains 11 %); of 640:
// 880 : 787, 880 : 813, 744 : 730, 620 : 621, 529 : 585. Two to eight elements of different lengths, 512
// keys at most: 832-883 : 767-806.
constexpr int kAfShortBlocks = 2, kAfShortBlocksPadded = 4;
constexpr float kAfRescale = 8.0f;  // log2 of the growth of a row's maximum that forces a rescale
// fp16 probabilities are held times 2^7 (2^15 at most with the above): what many keys weigh together
// may be a good part of a row although each has less than fp16's smallest 2^-25 of the largest.
constexpr float kAfUpF16 = 7.0f;

// Tensor memory columns: the two tiles' scores (their probabilities over them), their outputs.
constexpr int kAfS = 0, kAfO = 256;

// How a launch uses its units: two tiles with long runs of shared keys; the same with few key
// blocks, where the next queries need the room more than further keys; or one tile's rows twice,
// over two parts of the keys, and the same with 32 rows at most (single tokens), whose queries take
// a quarter of the room: the products read on past a slot's rows, into rows that nobody looks at.
enum AfMode { kAfLong = 0, kAfShort = 1, kAfPaired = 2, kAfToken = 3 };
constexpr int kAfTokenRows = 32;

template <int DP, int MODE, bool WIN>
struct AfSmem {
    static constexpr int kTile = kAttnRows * DP * 2;  // a tile of 128 rows; a block of 128 keys
    static constexpr int kHalf = kAttnRows * 128;     // its part of 64 columns
    static constexpr bool kPaired = MODE == kAfPaired || MODE == kAfToken;
    static constexpr int kSlotHalf = MODE == kAfToken ? kAfTokenRows * 128 : kHalf;
    static constexpr int kSlot = MODE == kAfToken ? kAfTokenRows * DP * 2 : kTile;
    static constexpr int kSlots =
        DP == 64 || MODE == kAfToken ? 4 : MODE == kAfLong ? 3 : MODE == kAfShort ? 4 : 2;
    static constexpr int kStages = DP == 64 ? 8 : MODE == kAfToken ? 6 : 7 - kSlots;
    // Registers a thread: 384 x 168 at launch = 256 x 216 + 128 x 72 = 256 x 208 + 128 x 88 (what
    // the roles take without spills)
    static constexpr int kRegsSoftmax = kPaired ? 208 : 216;
    static constexpr int kRegsOther = kPaired ? 88 : 72;
    // Units known at a time: a few, so that the next one's copies start early; single tokens the one
    // at work and the next, so that CTAs do not pile up what others could take (with four, 576 units
    // on 152 CTAs ended between 26 and 129 us).
    // (two at least: the softmax threads hold a record until their unit's end, and the products ask for the
    // next one before. Short windowed units too: the prompt of window 2,048 156 us with two, 158.5 with four.)
    static constexpr int kUnitSlots = kPaired || WIN ? 2 : kAfMaxUnitSlots;
    static constexpr int kQ = kAfBarBytes;  // barriers first
    static constexpr int kRing = kQ + kSlots * kSlot;
    static constexpr int kTotal = kRing + kStages * kTile;
    static_assert(kTotal + 1024 <= kSmemPerCtaMax, "shared memory");  // and room to align the base
};

template <bool WIN>
struct AfUnit : AttnBlocks<WIN> {
    int r, bb, kvh, sp;
    int tok0, tok1;  // first token of each tile
    int lo0, lo1;    // first key block of each tile
    int n0, n1;      // key blocks of each tile
    int len;         // keys of the batch element that any row sees
    int pos0;        // position of query token 0; beyond every key when not causal
    __device__ __forceinline__ int n(int k) const { return k ? n1 : n0; }
    __device__ __forceinline__ int lo(int k) const { return k ? lo1 : lo0; }
    __device__ __forceinline__ int tok(int k) const { return k ? tok1 : tok0; }
    __device__ __forceinline__ int most() const { return max(n0, n1); }
};

template <bool WIN>
struct AfBars {
    uint64_t u_full[kAfMaxUnitSlots], u_empty[kAfMaxUnitSlots];  // unit records
    uint64_t q_full[4], q_empty[4];  // query tile landed; its rows are written
    uint64_t s_full[2];              // scores complete
    uint64_t p_half[2], p_ready[2];  // half of the probabilities (and a rescaled O) written; all
    uint64_t o_full[2], o_free[2];   // output complete; read out
    uint64_t kv_full[8], kv_empty[8];
    uint64_t clean[8];               // rows past the last key zeroed
    uint64_t drain, steal;
    uint4 answer;
    uint32_t tmem;
    CtaLife life;
    AfUnit<WIN> unit[kAfMaxUnitSlots];  // r < 0: no more
};
static_assert(sizeof(AfBars<true>) <= kAfBarBytes, "barriers");

// Key blocks that the tile of tokens from `tok` on sees; with a window, those of the unit's list up to
// its last key (of two tiles of tokens the second's window may begin a block later: masked).
template <bool WIN>
__device__ __forceinline__ int af_blocks(const AttnFwdArgs& a, const AfUnit<WIN>& t, int64_t tok)
{
    const int64_t last = min(tok + a.tile_tokens, a.s.Sq) - 1;
    const int64_t keys = min(int64_t(t.len), t.pos0 + last + 1);
    if (tok >= a.s.Sq || keys <= 0) return 0;
    if constexpr (WIN) return (t.rows(a.s, keys) + kAttnRows - 1) / kAttnRows;
    return int((keys + kAttnRows - 1) / kAttnRows);
}

template <bool WIN>
__device__ __forceinline__ AfUnit<WIN> af_unit(const AttnFwdArgs& a, int64_t u)
{
    const AttnShape& s = a.s;
    AfUnit<WIN> t;
    const int64_t v = a.splits == 1 ? u : div_fast(u, a.splits);
    t.sp = int(u - v * a.splits);
    int64_t h, qb;
    attn_order(a.order, v, &h, &qb);
    if (s.causal) qb = a.order.blocks - 1 - qb;  // the longest rows first
    int r = 0;
    while (r + 1 < s.W && h >= s.head_begin[r + 1]) ++r;
    t.r = r;
    const int local = int(h) - s.head_begin[r];
    t.bb = local / s.m[r];
    t.kvh = local - t.bb * s.m[r];
    int64_t len, pos0;
    attn_limits(s, t.bb, &len, &pos0);
    t.len = int(len);
    t.pos0 = int(pos0);
    if (!WIN && a.paired) {
        t.tok0 = t.tok1 = 0;
        const int total = af_blocks(a, t, 0);
        const int per = (total + a.parts - 1) / a.parts;
        t.lo0 = 2 * t.sp * per;
        t.lo1 = t.lo0 + per;
        t.n0 = max(0, min(total - t.lo0, per));
        t.n1 = max(0, min(total - t.lo1, per));
    } else {
        const int64_t tok = qb * 2 * a.tile_tokens;
        t.tok0 = int(tok);
        t.tok1 = int(tok + a.tile_tokens);
        if constexpr (WIN)  // from the first row's window on
            t.set(s, max(int64_t(0), min(len, pos0 + tok + 1 - s.window)), len);
        const int b0 = af_blocks(a, t, tok), b1 = af_blocks(a, t, tok + a.tile_tokens);
        const int total = max(b0, b1);
        const int per = (total + a.splits - 1) / a.splits;
        t.lo0 = t.lo1 = t.sp * per;
        t.n0 = max(0, min(b0 - t.lo0, per));
        t.n1 = max(0, min(b1 - t.lo1, per));
    }
    return t;
}

// A warp's (or thread's) way through the CTA's units.
template <int SLOTS, bool WIN>
struct AfUnits {
    AfBars<WIN>* bars;
    StageRing ring;
    // The next unit; false: none, or the CTA has given up. WARP: called by a whole warp.
    template <bool WARP>
    __device__ __forceinline__ bool next(AfUnit<WIN>* t)
    {
        bool ok = wait_or_dead(&bars->u_full[ring.s], ring.phase, &bars->life);
        if (WARP) ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        *t = bars->unit[ring.s];
        if (t->r < 0) return false;
        release<WARP>();
        return true;
    }
    // The same without giving its record back yet (release does): it can be read again.
    __device__ __forceinline__ bool peek()
    {
        const bool ok = wait_or_dead(&bars->u_full[ring.s], ring.phase, &bars->life);
        return __all_sync(0xffffffffu, ok) && bars->unit[ring.s].r >= 0;
    }
    __device__ __forceinline__ const AfUnit<WIN>& record() const { return bars->unit[ring.s]; }
    template <bool WARP>
    __device__ __forceinline__ void release()
    {
        if (WARP) __syncwarp();
        if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(&bars->u_empty[ring.s]);
        ring.next(SLOTS);
    }
};

// Where a tile's row goes: its output, its log-sum-exp (or its part's), whether there is such a row.
struct AfRow {
    int64_t tok, o, part;  // token; byte offset in the rank's output; row of the part arrays
    float* lse;
    bool valid;
};

template <bool WIN>
__device__ __forceinline__ AfRow af_row(const AttnFwdArgs& a, const AfUnit<WIN>& t, int tile, int tok_in,
                                        int head_in)
{
    const AttnShape& s = a.s;
    AfRow r;
    r.tok = int64_t(t.tok(tile)) + tok_in;
    r.valid = tok_in < a.tile_tokens && r.tok < s.Sq;
    const int head = t.kvh * s.group + head_in;
    const int64_t row = (int64_t(t.bb) * s.n[t.r] + head) * s.Sq + r.tok;
    r.o = ((int64_t(t.bb) * s.Sq + r.tok) * s.n[t.r] + head) * s.d * 2;
    r.part = (a.paired ? 2 * t.sp + tile : t.sp) * s.row_begin[s.W] + s.row_begin[t.r] + row;
    r.lse = a.parts == 1 ? a.lse[t.r] + row : a.part_lse + r.part;
    return r;
}

// A row that sees no key (or no key of its part, which then has no output).
template <bool WIN>
__device__ __forceinline__ void af_empty_row(const AttnFwdArgs& a, const AfUnit<WIN>& t, const AfRow& r)
{
    if (!r.valid) return;
    *r.lse = -INFINITY;
    if (a.parts == 1)
        for (int c = 0; c < a.s.d * 2; c += 16) st_v4(a.o[t.r] + r.o + c, make_uint4(0, 0, 0, 0));
}

// The order in which a CTA's blocks of keys and values come, the products' own: block(value, t, key
// block) for every stage of the ring, and queries(t) for a unit's query tiles, after its first keys
// (a slot for them may have to wait for the unit before to finish, which those keys must not).
// Both return false to stop.
template <bool PAIRED, int SLOTS, bool WARP, bool WIN, class Queries, class Block>
__device__ __forceinline__ void af_walk(AfBars<WIN>* bars, Queries queries, Block block)
{
    AfUnits<SLOTS, WIN> units{bars};
    AfUnit<WIN> t;
    bool live = units.template next<WARP>(&t);
    while (live) {
        const int n = t.most();
        if constexpr (PAIRED) {  // each tile has keys of its own
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (t.n(k) > 0 && !block(false, t, t.lo(k))) return;
            if (!queries(t)) return;
            for (int j = 0; j < n; ++j) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (j < t.n(k) && !block(true, t, t.lo(k) + j)) return;
                    if (j + 1 < t.n(k) && !block(false, t, t.lo(k) + j + 1)) return;
                }
            }
        } else {
            if (!block(false, t, t.lo0) || !queries(t)) return;
            for (int j = 0; j < n; ++j) {
                if (!block(true, t, t.lo0 + j)) return;
                if (j + 1 < n && !block(false, t, t.lo0 + j + 1)) return;
            }
        }
        live = units.template next<WARP>(&t);
    }
}

// Rows of a value block past the batch element's last key, where any of them can hold a value
// (past the tensor's end the copy itself writes zeros); kAttnRows: none.
template <bool WIN>
__device__ __forceinline__ int af_past(const AttnShape& s, const AfUnit<WIN>& t, int block)
{
    int past = t.len - block * kAttnRows;
    if constexpr (WIN) past += t.pad - t.begin;
    return past >= kAttnRows || t.len >= s.Skv ? kAttnRows : past;
}

// Whether a value block holds rows that warp 10 zeroes.
template <bool WIN>
__device__ __forceinline__ bool af_unclean(const AttnShape& s, const AfUnit<WIN>& t, int block)
{
    if constexpr (WIN) {
        const int2 b = t.between(s, t.pos0, block);
        if (b.y > b.x) return true;
    }
    return af_past(s, t, block) < kAttnRows;
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t below(int n)
{
    return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// PAGED: the keys lie in pages (with a window, that may be none).
template <int DP, bool F16, int MODE, bool WIN, bool PAGED>
__global__ void __launch_bounds__(kAfThreads, 1)
    attn_fwd_kernel(const __grid_constant__ AttnFwdArgs a)
{
    using L = AfSmem<DP, MODE, WIN>;
    using E = ElemT<F16>;
    constexpr int K = L::kStages, Q = L::kSlots;
    constexpr bool PAIRED = L::kPaired;
    static_assert((!WIN || !PAIRED) && (!PAGED || WIN), "few rows with a window: attention_paged.cu");
    using Unit = AfUnit<WIN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    AfBars<WIN>& bars = *reinterpret_cast<AfBars<WIN>*>(smem);
    volatile CtaLife* life = &bars.life;
    const AttnShape& s = a.s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (s.d + 15) / 16;      // steps of 16 along the head dimension
    const int halves = (s.d + 63) / 64;  // tiles of 64 columns

    if (threadIdx.x == 0) {
        for (int k = 0; k < L::kUnitSlots; ++k) {
            mbar_init(&bars.u_full[k], 1);
            mbar_init(&bars.u_empty[k], s.ragged ? 11 : 10);  // warps 0-9, and 10
        }
        for (int k = 0; k < Q; ++k) {
            mbar_init(&bars.q_full[k], 1);
            mbar_init(&bars.q_empty[k], 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars.s_full[t], 1);
            mbar_init(&bars.p_half[t], 4);
            mbar_init(&bars.p_ready[t], 4);
            mbar_init(&bars.o_full[t], 1);
            mbar_init(&bars.o_free[t], 4);
        }
        for (int k = 0; k < K; ++k) {
            mbar_init(&bars.kv_full[k], 1);
            mbar_init(&bars.kv_empty[k], s.ragged ? 2 : 1);  // the products, and warp 10
            mbar_init(&bars.clean[k], 1);
        }
        mbar_init(&bars.drain, 1);
        mbar_init(&bars.steal, 1);
        life_init(bars.life, s.wait_us, kAfThreads / 32);
        fence_barrier_init();
    }
    if (warp == kAfMmaWarp) tmem_alloc(&bars.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp >= kAfLoadWarp) {
        regs_shrink<L::kRegsOther>();
        if (warp == kAfLoadWarp && (PAGED || lane == 0)) {  // (pages: a lane each)
            StageRing ring;
            StageRing slots;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool there = wait_or_dead(bar, parity, life);
                return PAGED ? bool(__all_sync(0xffffffffu, there)) : there;
            };
            int64_t issued = 0, tiles = 0;
            const uint32_t q_bytes = uint32_t(halves) * a.tile_tokens * s.group * 128u;
            const uint32_t kv_bytes = uint32_t(halves) * L::kHalf;
            auto queries = [&](const Unit& t) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (t.n(k) == 0) continue;
                    if (tiles >= Q && !wait(&bars.q_empty[slots.s], slots.phase ^ 1u)) return false;
                    if (!PAGED || lane == 0) {
                        mbar_arrive_expect_tx(&bars.q_full[slots.s], q_bytes);
                        for (int h = 0; h < halves; ++h)
                            tensor_g2s_4d(smem + L::kQ + slots.s * L::kSlot + h * L::kSlotHalf,
                                          &a.qmap[t.r], 64 * h, t.kvh * s.group, t.tok(k), t.bb,
                                          &bars.q_full[slots.s]);
                    }
                    ++tiles;
                    slots.next(Q);
                }
                return true;
            };
            // Pages: where this lane's rows of a block lie, for its keys and then its values.
            int page = 0, row = 0;
            bool needed = false;
            auto look = [&](const Unit& t, int at) {
                if constexpr (PAGED) {
                    const int v = at * kAttnRows + lane * a.pages.box, key = t.key(v);
                    // (a list from key 0 on holds keys between the first tokens and the unit's first window)
                    const int64_t first = t.pos0 + int64_t(t.tok0) + 1 - s.window;
                    needed = lane * a.pages.box < kAttnRows && key < (v < t.pad ? s.sinks : t.len) &&
                             (key < s.sinks || int64_t(key) + a.pages.box > first);
                    page = a.pages.pages;  // beyond the pool a copy writes zeros
                    row = 0;
                    if (needed) {
                        const int p = int(uint32_t(key) / uint32_t(a.pages.page));
                        page = a.pages.table[int64_t(t.bb) * a.pages.table_pages + p];
                        row = key - p * a.pages.page;
                    }
                }
            };
            auto block = [&](bool value, const Unit& t, int at) {
                if (PAGED && !value && at == t.lo0) look(t, at);
                if (issued >= K && !wait(&bars.kv_empty[ring.s], ring.phase ^ 1u)) return false;
                if constexpr (PAGED) {
                    if (lane == 0) mbar_arrive_expect_tx(&bars.kv_full[ring.s], kv_bytes);
                    __syncwarp();
                    if (needed && (page < 0 || page >= a.pages.pages))
                        atomicOr(&g_attn_fwd_status, kStatusBadPage);
                    if (lane * a.pages.box < kAttnRows)
                        for (int h = 0; h < halves; ++h)
                            tensor_g2s_4d(smem + L::kRing + ring.s * L::kTile + h * L::kHalf +
                                              lane * a.pages.box * 128,
                                          value ? &a.vmap[t.r] : &a.kmap[t.r], 64 * h, t.kvh, row, page,
                                          &bars.kv_full[ring.s]);
                    __syncwarp();
                    if (lane == 0) life->loads = uint32_t(issued + 1);
                    ++issued;
                    ring.next(K);
                    if (value) look(t, at + 1);  // (a block ahead)
                    return true;
                }
                mbar_arrive_expect_tx(&bars.kv_full[ring.s], kv_bytes);
                attn_load_keys<WIN, L::kHalf>(
                    smem + L::kRing + ring.s * L::kTile, halves, value ? &a.vmap[t.r] : &a.kmap[t.r],
                    value ? &a.vmap_sink[t.r] : &a.kmap_sink[t.r],
                    value ? &a.vmap_rest[t.r] : &a.kmap_rest[t.r], t, t.kvh, at, t.bb,
                    &bars.kv_full[ring.s]);
                life->loads = uint32_t(++issued);
                ring.next(K);
                return true;
            };
            af_walk<PAIRED, L::kUnitSlots, PAGED>(&bars, queries, block);
            // leave no copy into this CTA's shared memory in flight
            // (called by one lane or by all)
            for (int64_t k = max(int64_t(0), issued - K); k < issued; ++k)
                if (!mbar_wait_bounded(&bars.kv_full[k % K], uint32_t((k / K) & 1)))
                    atomicOr(&g_attn_fwd_status, kStatusDrainTimeout);
            for (int64_t k = max(int64_t(0), tiles - Q); k < tiles; ++k)
                if (!mbar_wait_bounded(&bars.q_full[k % Q], uint32_t((k / Q) & 1)))
                    atomicOr(&g_attn_fwd_status, kStatusDrainTimeout);
        } else if (warp == kAfCleanWarp && s.ragged) {
            // A masked probability is zero, but zero times whatever lies past the last key may be
            // NaN: a value block's rows past it become zeros before its product.
            StageRing ring;
            af_walk<PAIRED, L::kUnitSlots, true>(
                &bars, [](const Unit&) { return true; },
                [&](bool value, const Unit& t, int at) {
                    const int past = value ? af_past(s, t, at) : kAttnRows;
                    int2 between = make_int2(0, 0);
                    if constexpr (WIN)
                        if (value) between = t.between(s, t.pos0, at);
                    if (!__all_sync(0xffffffffu,
                                    wait_or_dead(&bars.kv_full[ring.s], ring.phase, life)))
                        return false;
                    if (past < kAttnRows || between.y > between.x) {
                        for (int h = 0; h < halves; ++h) {
                            uint8_t* rows = smem + L::kRing + ring.s * L::kTile + h * L::kHalf;
                            for (int w = past * 8 + lane; w < kAttnRows * 8; w += 32)
                                st_shared_v4(rows + w * 16, make_uint4(0, 0, 0, 0));
                            if constexpr (WIN)
                                for (int w = between.x * 8 + lane; w < between.y * 8; w += 32)
                                    st_shared_v4(rows + w * 16, make_uint4(0, 0, 0, 0));
                        }
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.clean[ring.s]);
                    }
                    // every stage waits for this warp, so that it neither runs ahead of the ring
                    // nor falls a turn behind
                    if (lane == 0) mbar_arrive(&bars.kv_empty[ring.s]);
                    ring.next(K);
                    return true;
                });
        } else if (warp == kAfMmaWarp && elect_one()) {
            const uint32_t id_s = tc_idesc(F16, kAttnRows, false);
            const uint32_t id_o = tc_idesc(F16, 16 * nk, true);
            const uint64_t q_desc = tc_desc_k(smem_u32(smem + L::kQ));
            const uint64_t k_desc = tc_desc_k(smem_u32(smem + L::kRing));
            const uint64_t v_desc = tc_desc_mn(smem_u32(smem + L::kRing), L::kHalf);
            StageRing ring, slots;
            int slot[2] = {0, 0};  // of each tile's queries
            uint32_t uses[2] = {0, 0}, blocks[2] = {0, 0};
            uint32_t cleaned = 0;  // parity of each stage's `clean`
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return ok = ok && wait_or_dead(bar, parity, life);
            };
            auto scores = [&](int k, int stage) {  // S_k = Q_k K^T
                const uint64_t qd = q_desc + slot[k] * (L::kSlot >> 4);
                const uint64_t kd = k_desc + stage * (L::kTile >> 4);
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    if (ks >= nk) break;
                    tc_mma_ss(tmem + kAfS + k * 128,
                              qd + (((ks >> 2) * L::kSlotHalf + (ks & 3) * 32) >> 4),
                              kd + (((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4), id_s, ks > 0);
                }
                tc_commit(&bars.s_full[k]);
            };
            auto first_scores = [&](int k, int stage) {  // of a unit, its tiles in order
                if (!wait(&bars.q_full[slots.s], slots.phase)) return;
                slot[k] = slots.s;
                slots.next(Q);
                tc_fence_after();
                scores(k, stage);
            };
            auto output = [&](const Unit& t, int k, int stage, int j) {  // O_k += P_k V
                wait(&bars.p_half[k], blocks[k] & 1);
                if (j == 0 && uses[k] > 0) wait(&bars.o_free[k], (uses[k] - 1) & 1);
                if (!ok) return;
                const uint64_t vd = v_desc + stage * (L::kTile >> 4);
                auto half = [&](int from) {
                    tc_fence_after();
#pragma unroll
                    for (int ks = from; ks < from + 4; ++ks)
                        tc_mma_ts(tmem + kAfO + k * 128, tmem + kAfS + k * 128 + ks * 8,
                                  vd + ks * (2048 >> 4), id_o, j > 0 || ks > 0);
                };
                half(0);
                if (!wait(&bars.p_ready[k], blocks[k] & 1)) return;
                half(4);
                ++blocks[k];
                if (j + 1 == t.n(k)) {
                    tc_commit(&bars.o_full[k]);
                    ++uses[k];
                }
            };
            auto stage_ready = [&]() { return wait(&bars.kv_full[ring.s], ring.phase); };
            auto values_ready = [&](const Unit& t, int at) {
                stage_ready();
                if (s.ragged && af_unclean(s, t, at)) {
                    wait(&bars.clean[ring.s], (cleaned >> ring.s) & 1);
                    cleaned ^= 1u << ring.s;
                }
                return ok;
            };
            auto unit_scores = [&](const Unit& t) {  // a paired unit's first scores
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (t.n(k) == 0 || !stage_ready()) continue;
                    first_scores(k, ring.s);
                    tc_commit(&bars.kv_empty[ring.s]);
                    ring.next(K);
                }
            };
            AfUnits<L::kUnitSlots, WIN> units{&bars};
            Unit t, next;
            bool live = units.template next<false>(&t);
            if (live) {
                if constexpr (PAIRED) {
                    unit_scores(t);
                } else if (stage_ready()) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (t.n(k) > 0) first_scores(k, ring.s);
                    tc_commit(&bars.kv_empty[ring.s]);
                    ring.next(K);
                }
            }
            while (live && ok) {
                bool more = false;
                const int n = t.most();
                for (int j = 0; ok && j < n; ++j) {
                    // (asked for as late as it is needed: see kUnitSlots)
                    if (j + 1 == n) more = units.template next<false>(&next);
                    if constexpr (PAIRED) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (j < t.n(k)) {
                                if (!values_ready(t, t.lo(k) + j)) break;
                                output(t, k, ring.s, j);
                                tc_commit(&bars.kv_empty[ring.s]);
                                ring.next(K);
                            }
                            if (j + 1 < t.n(k)) {
                                if (!stage_ready()) break;
                                scores(k, ring.s);
                                tc_commit(&bars.kv_empty[ring.s]);
                                ring.next(K);
                            }
                        }
                    } else {
                        const bool last = j + 1 == n;
                        const int vs = ring.s;
                        if (!values_ready(t, t.lo0 + j)) break;
                        ring.next(K);
                        const int ks = ring.s;
                        const bool any = !last || more;
                        if (any) {
                            if (!stage_ready()) break;
                            ring.next(K);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (j < t.n(k)) output(t, k, vs, j);
                            if (!ok) break;
                            if (j + 1 < t.n(k))
                                scores(k, ks);
                            else if (last && more && next.n(k) > 0)
                                first_scores(k, ks);
                        }
                        tc_commit(&bars.kv_empty[vs]);
                        if (any) tc_commit(&bars.kv_empty[ks]);
                    }
                }
                if (PAIRED && more) unit_scores(next);
                t = next;
                live = more;
            }
            // every product complete before tensor memory is given back
            tc_commit(&bars.drain);
            if (!mbar_wait_bounded(&bars.drain, 0)) atomicOr(&g_attn_fwd_status, kStatusDrainTimeout);
        }
        else if (warp == kAfUnitWarp) {
            StageRing ring;
            bool ok = true;
            int64_t made = 0;
            auto room = [&]() {  // before a unit is taken, not with one in hand
                if (made >= L::kUnitSlots)
                    ok = __all_sync(0xffffffffu,
                                    wait_watching(&bars.u_empty[ring.s], ring.phase ^ 1u, life));
                return ok;
            };
            auto publish = [&](const Unit& t) {
                if (lane == 0) {
                    bars.unit[ring.s] = t;
                    mbar_arrive(&bars.u_full[ring.s]);
                }
                __syncwarp();
                ++made;
                ring.next(L::kUnitSlots);
            };
            Unit t;
            AttnUnitSource source{a.units, &bars.answer, &bars.steal, life};
            for (int64_t u; room() && (u = source.next()) >= 0;) {
                t = af_unit<WIN>(a, u);
                if (t.most() > 0) {
                    publish(t);
                } else {  // nothing to do but say so (the other warps see units with work only)
                    for (int i = lane; i < 2 * kAttnRows; i += 32) {
                        const int tile = i / kAttnRows, row = i % kAttnRows;
                        const int tok_in = row / s.group;
                        af_empty_row(a, t, af_row(a, t, tile, tok_in, row - tok_in * s.group));
                    }
                }
            }
            t.r = -1;
            if (ok) publish(t);
        }
        __syncwarp();
    } else {  // softmax: tile w = warp / 4, one row a thread
        regs_grow<L::kRegsSoftmax>();
        const int tile = warp >> 2;
        const int row = threadIdx.x & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t s_at = tmem + lanes + kAfS + tile * 128;
        const uint32_t o_at = tmem + lanes + kAfO + tile * 128;
        const int tok_in = row / s.group, head_in = row - tok_in * s.group;
        const float sl2 = s.scale * 1.4426950408889634f;  // scores to powers of two
        constexpr float kUp = F16 ? kAfUpF16 : 0.0f;
        const int rows = a.tile_tokens * s.group;         // of a tile
        uint32_t uses = 0, blocks = 0;
        bool ok = true;
        auto all = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_or_dead(bar, parity, life));
        };
        auto arrive = [&](uint64_t* bar) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        AfUnits<L::kUnitSlots, WIN> units{&bars};
        StageRing slots;
        while (ok && units.peek()) {
            // What the loop over the blocks does not need is read again after it: a row's scores
            // take 128 registers.
            int slot = 0, n, left;  // of this tile's queries; its blocks; keys seen from its first
            // with a window: where the row's begins in the tile's blocks, where the first tokens end, the
            // blocks up to any row's of the warp
            int low = 0, sinks = 0, edge = 0;
            {
                const Unit& t = units.record();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (t.n(k) == 0) continue;
                    if (k == tile) slot = slots.s;
                    slots.next(Q);
                }
                n = t.n(tile);
                if (n == 0) {
                    af_empty_row(a, t, af_row(a, t, tile, tok_in, head_in));
                    units.template release<true>();
                    continue;
                }
                const int64_t seen = min(int64_t(t.len), t.pos0 + int64_t(t.tok(tile)) + tok_in + 1);
                if constexpr (WIN) {
                    const int64_t first = t.pos0 + int64_t(t.tok(tile)) + tok_in + 1 - s.window;
                    low = int(max(int64_t(0), min(int64_t(t.len), first) - t.begin)) + t.pad -
                          t.lo(tile) * kAttnRows;
                    left = t.rows(s, seen) - t.lo(tile) * kAttnRows;
                    sinks = s.sinks - t.lo(tile) * kAttnRows;
                    edge = (__reduce_max_sync(0xffffffffu, low) + kAttnRows - 1) >> 7;
                } else {
                    left = int(max(int64_t(-1), seen - int64_t(t.lo(tile)) * kAttnRows));
                }
            }
            float m = -INFINITY, l = 0.0f;
            if (PAIRED && (warp & 3) * 32 >= rows) {  // none of the tile's rows: only keep step
                for (int j = 0; j < n; ++j) {
                    ok = all(&bars.s_full[tile], blocks & 1);
                    if (!ok) break;
                    ++blocks;
                    arrive(&bars.p_half[tile]);
                    arrive(&bars.p_ready[tile]);
                }
                if (ok) ok = all(&bars.o_full[tile], uses & 1);
                if (!ok) break;
                ++uses;
                if (lane == 0) {
                    mbar_arrive(&bars.o_free[tile]);
                    mbar_arrive(&bars.q_empty[slot]);
                }
                units.template release<true>();
                continue;
            }
            for (int j = 0; j < n; ++j, left -= kAttnRows) {
                ok = all(&bars.s_full[tile], blocks & 1);
                if (!ok) break;
                ++blocks;
                tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(s_at + q * 32, x[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_wait_ld(x[q]);
                if constexpr (WIN) {
                    // keys in view: below the row's last, but those between the first tokens and its window
                    const int from = sinks - j * kAttnRows, to = low - j * kAttnRows;
                    const bool begins = j < edge && from < kAttnRows;
                    if (__any_sync(0xffffffffu, left < kAttnRows) || begins) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t see = below(left - q * 32);
                            if (begins) see &= below(from - q * 32) | ~below(to - q * 32);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(see >> c & 1u)) x[q][c] = 0xFF800000u;  // -infinity
                        }
                    }
                } else if (__any_sync(0xffffffffu, left < kAttnRows)) {
                    const int seen = max(0, left);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (q * 32 + c >= seen) x[q][c] = 0xFF800000u;  // -infinity
                }
                float mx[4] = {m, m, m, m};
#pragma unroll
                for (int c = 0; c < 32; c += 2)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mx[q] = max3(mx[q], __uint_as_float(x[q][c]), __uint_as_float(x[q][c + 1]));
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                const bool grow = (top - m) * sl2 > kAfRescale;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2((m - top) * sl2) : 1.0f;
                    if (grow) m = top;
                    l *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < DP / 32; ++c) {
                            uint32_t y[32];
                            tmem_ld32(o_at + c * 32, y);
                            tmem_wait_ld(y);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                            tmem_st32(o_at + c * 32, y);
                        }
                    }
                }
                const float base = (m == -INFINITY ? 0.0f : -m * sl2) + kUp;
                const float2 k2 = make_float2(sl2, sl2), b2 = make_float2(base, base);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 e = __ffma2_rn(make_float2(__uint_as_float(x[q][2 * i]),
                                                          __uint_as_float(x[q][2 * i + 1])),
                                              k2, b2);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                        p[i] = E::pack(e.x, e.y);
                    }
                    tmem_st16(s_at + q * 16, p);
                    if (q == 1) arrive(&bars.p_half[tile]);
                }
                arrive(&bars.p_ready[tile]);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (!ok) break;
            ok = all(&bars.o_full[tile], uses & 1);
            if (!ok) break;
            tc_fence_after();
            const Unit& t = units.record();
            const AfRow to = af_row(a, t, tile, tok_in, head_in);
            const bool whole = a.parts == 1;
            uint8_t* o = a.o[t.r];
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // NaN stays NaN
            if (to.valid)
                *to.lse = l == 0.0f ? -INFINITY : m * s.scale + (logf(l) - kUp * 0.69314718056f);
            float* o_part = a.part_o + to.part * s.d;
            uint8_t* stage = smem + L::kQ + slot * L::kSlot;  // the queries are done with
#pragma unroll 1  // (rolled: short units go round all of this kernel's code all the time)
            for (int c = 0; c < DP / 32; ++c) {
                uint32_t y[32];
                tmem_ld32(o_at + c * 32, y);
                tmem_wait_ld(y);
                if (c == DP / 32 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.o_free[tile]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // eight columns
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(y[8 * i + k]) * inv;
                    if (whole) {
                        const int word = (c & 1) * 4 + i;
                        st_shared_v4(stage + (c >> 1) * L::kHalf + row * 128 +
                                         ((word ^ (row & 7)) << 4),
                                     make_uint4(E::pack(v[0], v[1]), E::pack(v[2], v[3]),
                                                E::pack(v[4], v[5]), E::pack(v[6], v[7])));
                    } else if (to.valid && c * 32 + i * 8 < s.d) {
                        float4* dst = reinterpret_cast<float4*>(o_part + c * 32 + i * 8);
                        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
            if (whole) {  // this warp's 32 rows, 8 lanes a row's 64 columns
                // (before the stores: a fence behind them waits for them, some microseconds)
                fence_proxy_async_shared();
                __syncwarp();
                const int64_t at = to.valid ? to.o : -1;
                const int word = lane & 7;
#pragma unroll 2
                for (int i = 0; i < 8; ++i) {
                    const int rr = i * 4 + (lane >> 3);
                    const int64_t off = __shfl_sync(0xffffffffu, at, rr);
#pragma unroll
                    for (int h = 0; h < DP / 64; ++h) {
                        if (off < 0 || h * 64 + word * 8 >= s.d) continue;
                        st_v4(o + off + h * 128 + word * 16,
                              ld_shared_v4(stage + h * L::kHalf + ((warp & 3) * 32 + rr) * 128 +
                                           ((word ^ (rr & 7)) << 4)));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.q_empty[slot]);
            units.template release<true>();
            ++uses;
        }
    }
    life_end(bars.life, warp == kAfUnitWarp);
    let_next_start();
    __syncthreads();
    if (threadIdx.x == 0 && life_status(bars.life) != 0)
        atomicOr(&g_attn_fwd_status, life_status(bars.life));
    if (warp == kAfMmaWarp) tmem_free(tmem);
}

// Joins the parts of the keys: one warp a row; lane c holds columns 4c .. 4c + 3 of the outputs, and
// the weights of parts c, c + 32, ... Every part's lse is on its way at once, then the outputs of
// four parts at a time (one after the other, each waited for the memory's latency).
template <bool F16>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnFwdArgs a)
{
    using E = ElemT<F16>;
    const AttnShape& s = a.s;
    const int64_t rows = s.row_begin[s.W];
    const int lane = threadIdx.x & 31;
    constexpr int kEach = kAfMaxParts / 32;
    wait_for_previous();
    for (int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5); row < rows;
         row += int64_t(gridDim.x) * 4) {
        float w[kEach], top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int p = i * 32 + lane;
            w[i] = p < a.parts ? a.part_lse[p * rows + row] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) top = fmaxf(top, w[i]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
#pragma unroll
        for (int i = 0; i < kEach; ++i) {  // (NaN stays NaN)
            w[i] = w[i] == -INFINITY ? 0.0f : expf(w[i] - top);
            sum += w[i];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            for (int p0 = 0; p0 < 32 && i * 32 + p0 < a.parts; p0 += 4) {
                float4 o[4];
                float f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[k] = __shfl_sync(0xffffffffu, w[i], p0 + k);
                    o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    // an empty part (weight 0) wrote no output
                    if (f[k] != 0.0f && lane * 4 < s.d)
                        o[k] = *reinterpret_cast<const float4*>(
                            a.part_o + ((i * 32 + p0 + k) * rows + row) * s.d + lane * 4);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc.x = fmaf(f[k], o[k].x, acc.x);
                    acc.y = fmaf(f[k], o[k].y, acc.y);
                    acc.z = fmaf(f[k], o[k].z, acc.z);
                    acc.w = fmaf(f[k], o[k].w, acc.w);
                }
            }
        }
        int r = 0;
        while (r + 1 < s.W && row >= s.row_begin[r + 1]) ++r;
        const int64_t local = row - s.row_begin[r];  // (batch * n_r + head) * Sq + token
        const int64_t bh = div_fast(local, s.Sq), tok = local - bh * s.Sq;
        const int64_t bb = bh / s.n[r], head = bh - bb * s.n[r];
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (lane * 4 < s.d)
            st_v2(a.o[r] + (((bb * s.Sq + tok) * s.n[r] + head) * s.d + lane * 4) * 2,
                  E::pack(acc.x * inv, acc.y * inv), E::pack(acc.z * inv, acc.w * inv));
        if (lane == 0) a.lse[r][local] = sum == 0.0f ? top : top + logf(sum);
    }
}

template <int DP, bool F16, int MODE, bool WIN, bool PAGED>
static cudaError_t af_launch_mode(const AttnFwdArgs& a, cudaStream_t stream, int device, int64_t cap,
                                  int sm_count)
{
    static std::atomic<unsigned long long> raised{0};
    const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0;
    constexpr int smem = AfSmem<DP, MODE, WIN>::kTotal + 1024;
    if (bit && !(raised.load() & bit)) {
        cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<DP, F16, MODE, WIN, PAGED>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit);
    }
    attn_fwd_kernel<DP, F16, MODE, WIN, PAGED>
        <<<attn_ctas(a.units, cap, sm_count), kAfThreads, smem, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.parts == 1) return e;
    int64_t blocks = (a.s.row_begin[a.s.W] + 3) / 4;
    if (blocks > 1 << 16) blocks = 1 << 16;
    return attn_launch_early(attn_join_kernel<F16>, unsigned(blocks < cap ? blocks : cap), 128, 0,
                             stream, a, cap == kAttnMostCtas);
}

// By the head dimension and the type.
template <int MODE, bool WIN, bool PAGED>
static cudaError_t af_launch_types(const AttnFwdArgs& a, cudaStream_t stream, int device, int64_t cap,
                                   int sm_count)
{
    if (a.s.d <= 64)
        return a.s.f16 ? af_launch_mode<64, true, MODE, WIN, PAGED>(a, stream, device, cap, sm_count)
                       : af_launch_mode<64, false, MODE, WIN, PAGED>(a, stream, device, cap, sm_count);
    return a.s.f16 ? af_launch_mode<128, true, MODE, WIN, PAGED>(a, stream, device, cap, sm_count)
                   : af_launch_mode<128, false, MODE, WIN, PAGED>(a, stream, device, cap, sm_count);
}

// The word that this source file's kernels set.
static cudaError_t af_status(unsigned* status, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_attn_fwd_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_fwd_status, &zero, sizeof(unsigned));
}

}  // namespace uly
