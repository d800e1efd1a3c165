// attention_bwd.cu -- gradients of attention with the probabilities recomputed.
//
// With P_ij = exp(s_ij - lse_i) over visible keys, D_i = sum_c dO_ic O_ic, dP = dO V^T and
// dS = P (dP - D):  dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K. Keys shared by several
// query heads sum over them. Five products of 2 d flops per (row, key) cannot be done without.
//
// Three launches; the last two start before the one in front of them has ended. attn_bwd_stats_kernel writes each row's lse (in powers of two; +infinity where a
// row sees nothing or does not exist, which makes its P zero) and D in row-tile order, with fp16 the
// norms that give P and dS their place in its range as well (see ab_exponent: 2,047 causal tokens, 24
// heads over 8 of 64 take 189 us with them, 178 without). Then
// attn_bwd_kv_kernel holds a block of 128 keys and walks the row tiles that see it (dK, dV), and
// attn_bwd_q_kernel holds a tile of 128 rows and walks its key blocks (dQ). S and dP are computed
// by both, seven products in place of five: dQ is then summed in one accumulator in a fixed order,
// with no fp32 copy of it in memory, no atomics, and the same bits from run to run.
//
// Both are bound by the products; those with both operands in shared memory take about 107 cycles
// in place of 64. Measured at 16,380 tokens x 8 heads of 128: 2.58-2.60 ms, 1.06 PFLOP/s with five
// products counted (alone: dK, dV 1,440 us, 2,736 of whose 3,000 cycles a tile are products, dQ 960 us,
// statistics 12 us). One CTA per SM (640 threads): 16 warps turn scores into P and
// dS, each four the same 32 columns of the tile (16 warps rather than 8 with twice the columns: the
// chain from scores to P is what the products wait for, and more warps hide its latencies). Warp 16
// loads (swizzled tensor maps), one lane of warp 17 issues the products, which run on one operand
// while the threads work on the other; a unit's first scores follow the last unit's products
// without a gap. All accumulators are in tensor memory (fp32); P and dS go back to it rounded to
// the element type, over the columns they came from, and are A operands there. Warp 18 of the dQ
// kernel zeroes what a key block holds past a ragged batch element's last key, the one of the dK, dV
// kernel what rows that see no key hold. Warp 19 works out the units ahead.
// Roundings: P and dS to the element type (relative errors of half a step each, in sums of either
// sign), the gradients once; every sum, the statistics and the exponents are fp32.
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

static __device__ unsigned g_attn_bwd_status;

constexpr int kAbThreads = 640;
constexpr int kAbLoadWarp = 16, kAbMmaWarp = 17, kAbCleanWarp = 18, kAbUnitWarp = 19;
// Units known ahead of the slowest reader: one, so that CTAs do not pile up units others could take.
constexpr int kAbUnitSlots = 1;
constexpr int kAbStats = 2 * kAttnRows * 4;  // one tile's lse and D
template <bool F16>
constexpr int kAbStatArrays = F16 ? 3 : 2;  // a tile's arrays of row statistics

__device__ __forceinline__ void ab_head(const AttnShape& s, int64_t h, int* r, int* bb, int* kvh)
{
    int k = 0;
    while (k + 1 < s.W && h >= s.head_begin[k + 1]) ++k;
    const int local = int(h) - s.head_begin[k];
    *r = k;
    *bb = local / s.m[k];
    *kvh = local - *bb * s.m[k];
}

// The largest of all threads' values (256 of them), in every thread.
__device__ __forceinline__ float ab_block_max(float x, float* shared)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    x = shared[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) x = fmaxf(x, shared[w]);
    return x;
}

// Sum over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float ab_row_sum(float x)
{
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Half a tile of rows a CTA; LANES lanes a row, 8 columns each. Bound by reading O and dO. With fp16
// also the largest |v| of each block of keys, and what else bounds dS (see ab_exponent).
template <bool F16, int LANES>
__global__ void __launch_bounds__(256) attn_bwd_stats_kernel(const __grid_constant__ AttnBwdArgs a)
{
    using E = ElemT<F16>;
    const AttnShape& s = a.s;
    constexpr int kAtOnce = 256 / LANES, kTurns = kAttnRows / 2 / kAtOnce;
    __shared__ float shared[8];
    const int sub = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    let_next_start();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ready = 0;
    const int64_t halves = 2 * s.head_begin[s.W] * a.q_tiles;
    for (int64_t at = blockIdx.x; at < halves; at += gridDim.x) {
        const int64_t tile = at >> 1;
        const int row0 = int(at & 1) * (kAttnRows / 2) + slot;
        const int64_t h = div_fast(tile, a.q_tiles);
        int r, bb, kvh;
        ab_head(s, h, &r, &bb, &kvh);
        const int64_t tok0 = (tile - h * a.q_tiles) * a.tile_tokens;
        uint4 x[kTurns], y[kTurns];
        float lse[kTurns];
        bool valid[kTurns];
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {  // every load before the first use
            const int row = k * kAtOnce + row0;
            const int tok_in = row / s.group, head = kvh * s.group + row - tok_in * s.group;
            const int64_t tok = tok0 + tok_in;
            valid[k] = tok_in < a.tile_tokens && tok < s.Sq;
            x[k] = y[k] = make_uint4(0, 0, 0, 0);
            lse[k] = -INFINITY;
            if (valid[k] && sub * 8 < s.d) {
                const int64_t off =
                    ((int64_t(bb) * s.Sq + tok) * s.n[r] + head) * s.d * 2 + sub * 16;
                x[k] = ld_stream_v4(a.o[r] + off);
                y[k] = ld_stream_v4(a.go[r] + off);
            }
            if (valid[k] && sub == 0) lse[k] = a.lse[r][(int64_t(bb) * s.n[r] + head) * s.Sq + tok];
        }
        float most_g = 0.0f, most_d = 0.0f;
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const uint32_t xs[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            const uint32_t ys[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
            float sum = 0.0f, square = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum = fmaf(E::lo(xs[i]), E::lo(ys[i]), sum);
                sum = fmaf(E::hi(xs[i]), E::hi(ys[i]), sum);
                if (F16) {
                    square = fmaf(E::lo(ys[i]), E::lo(ys[i]), square);
                    square = fmaf(E::hi(ys[i]), E::hi(ys[i]), square);
                }
            }
            sum = ab_row_sum<LANES>(sum);
            if (F16) square = ab_row_sum<LANES>(square);
            if (sub == 0) {
                const bool none = lse[k] == -INFINITY;
                const float z = lse[k] * 1.4426950408889634f;
                float* out = a.stats + tile * kAbStatArrays<F16> * kAttnRows + k * kAtOnce + row0;
                out[0] = none ? INFINITY : F16 ? z - kAttnPBits : z;
                out[kAttnRows] = none ? 0.0f : sum;
                if (F16) {
                    const float norm = none ? 0.0f : sqrtf(square);
                    out[2 * kAttnRows] = norm;
                    most_g = fmaxf(most_g, norm);
                    most_d = fmaxf(most_d, none ? 0.0f : fabsf(sum));
                }
            }
        }
        if (F16) {
            most_g = ab_block_max(most_g, shared);
            most_d = ab_block_max(most_d, shared);
            if (threadIdx.x == 0) a.row_bounds[at] = make_float2(most_g, most_d);
        }
    }
    if (!F16) return;
    const int64_t blocks = a.kv_order.blocks, all = s.head_begin[s.W] * blocks;
    // (the CTAs after those with rows first)
    const int64_t from = (halves + gridDim.x - 1 - blockIdx.x) / gridDim.x * gridDim.x + blockIdx.x;
    for (int64_t at = from - halves; at < all; at += gridDim.x) {
        const int64_t h = div_fast(at, blocks), block = at - h * blocks;
        int r, bb, kvh;
        ab_head(s, h, &r, &bb, &kvh);
        int64_t len, pos0;
        attn_limits(s, bb, &len, &pos0);
        uint4 v[2 * kTurns];
#pragma unroll
        for (int k = 0; k < 2 * kTurns; ++k) {
            const int64_t key = block * kAttnRows + k * kAtOnce + slot;
            v[k] = make_uint4(0, 0, 0, 0);
            if (key < len && sub * 8 < s.d)
                v[k] = ld_stream_v4(a.v[r] + ((int64_t(bb) * s.Skv + key) * s.m[r] + kvh) * s.d * 2 +
                                    sub * 16);
        }
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < 2 * kTurns; ++k) {
            const uint32_t vs[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            float square = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                square = fmaf(E::lo(vs[i]), E::lo(vs[i]), square);
                square = fmaf(E::hi(vs[i]), E::hi(vs[i]), square);
            }
            most = fmaxf(most, ab_row_sum<LANES>(square));
        }
        most = ab_block_max(most, shared);
        if (threadIdx.x == 0) a.key_norms[at] = sqrtf(most);
    }
}

// fp16 holds its 11 bits between 6e-5 and 65,504 only, and dS = P (dP - D) is as small as 1 / keys times
// dO, or as large as dO v. So it is held times a power of two that a bound gives it:
// |dP_ij - D_i| <= |dO_i| |v_j| + |D_i|, and P <= 1. dQ's rows have one each, dK's sums run over rows
// and have one a unit (a key block with all the rows that see it); the gradients' last factor takes it
// out again. The exponent with bound 2^e below 2^15 (a zero bound, or one of infinities: any will do).
__device__ __forceinline__ int ab_exponent(float bound)
{
    const int x = (__float_as_int(bound) >> 23) - 127;
    return 14 - max(-80, min(x, 60));
}

__device__ __forceinline__ float ab_power(int e) { return __int_as_float((e + 127) << 23); }

// P (dP - D) of two columns; d is -D.
__device__ __forceinline__ float2 ab_ds(uint32_t p0, uint32_t p1, uint32_t y0, uint32_t y1, float2 d)
{
    return __fmul2_rn(make_float2(__uint_as_float(p0), __uint_as_float(p1)),
                      __fadd2_rn(make_float2(__uint_as_float(y0), __uint_as_float(y1)), d));
}

// N columns from `col` on of an accumulator's row, times f, to the row of d elements at `out`.
template <class E, int N>
__device__ __forceinline__ void ab_store(uint8_t* out, int col, int d, const uint32_t (&y)[N], float f)
{
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        if (col + i * 8 >= d) continue;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = E::pack(__uint_as_float(y[8 * i + 2 * k]) * f,
                           __uint_as_float(y[8 * i + 2 * k + 1]) * f);
        st_v4(out + (col + i * 8) * 2, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// The units ahead, worked out by one warp (publish) and read by the others (next). Units without
// work do not appear.
template <class Unit>
struct AbUnitBoard {
    uint64_t full[kAbUnitSlots], empty[kAbUnitSlots], steal;
    uint4 answer;
    Unit unit[kAbUnitSlots];  // n < 0: no more
};

template <class Unit>
__device__ __forceinline__ void ab_board_init(AbUnitBoard<Unit>& b, int readers)
{
    for (int k = 0; k < kAbUnitSlots; ++k) {
        mbar_init(&b.full[k], 1);
        mbar_init(&b.empty[k], readers);
    }
    mbar_init(&b.steal, 1);
}

template <class Unit>
struct AbUnits {
    AbUnitBoard<Unit>* board;
    volatile CtaLife* life;
    StageRing ring;
    // The next unit; false: none, or the CTA has given up. WARP: called by a whole warp.
    template <bool WARP>
    __device__ __forceinline__ bool next(Unit* t)
    {
        bool ok = wait_or_dead(&board->full[ring.s], ring.phase, life);
        if (WARP) ok = __all_sync(0xffffffffu, ok);
        if (ok) *t = board->unit[ring.s];
        if (!ok || t->n < 0) {
            t->n = 0;
            return false;
        }
        if (WARP) __syncwarp();
        if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(&board->empty[ring.s]);
        ring.next(kAbUnitSlots);
        return true;
    }
};

// The warp that works the units out: decode(u) gives a unit, idle(t) deals with one without work.
template <class Unit, class Decode, class Idle>
__device__ __forceinline__ void ab_publish(AbUnitBoard<Unit>& b, int64_t units, volatile CtaLife* life,
                                           Decode decode, Idle idle)
{
    StageRing ring;
    AttnUnitSource source{units, &b.answer, &b.steal, life};
    bool ok = true;
    for (int64_t made = 0;;) {
        if (made >= kAbUnitSlots)  // before a unit is taken, not with one in hand
            ok = __all_sync(0xffffffffu, wait_watching(&b.empty[ring.s], ring.phase ^ 1u, life));
        if (!ok) break;
        const int64_t u = source.next();
        Unit t;
        t.n = -1;
        if (u >= 0) {
            t = decode(u);
            if (t.n == 0) {
                idle(t);
                continue;
            }
        }
        if ((threadIdx.x & 31) == 0) {
            b.unit[ring.s] = t;
            mbar_arrive(&b.full[ring.s]);
        }
        __syncwarp();
        ++made;
        ring.next(kAbUnitSlots);
        if (u < 0) break;
    }
}

// ---- dK and dV ----------------------------------------------------------------------------------

// Tensor memory columns. S^T (then P^T) and dP^T (then dS^T): lanes are keys, columns rows of q.
constexpr int kBkS = 0, kBkDp = 128, kBkDv = 256, kBkDk = 384;

template <int DP>
struct BkSmem {
    static constexpr int kTile = kAttnRows * DP * 2;
    static constexpr int kHalf = kAttnRows * 128;
    static constexpr int kStages = DP == 128 ? 2 : 4;
    static constexpr int kK = 1024, kV = kK + kTile;
    static constexpr int kQ = kV + kTile;               // ring of q tiles
    static constexpr int kG = kQ + kStages * kTile;     // ring of dO tiles
    static constexpr int kStat = kG + kStages * kTile;  // ring of their lse and D
    static constexpr int kTotal = kStat + kStages * kAbStats;
    static_assert(kTotal + 1024 <= kSmemPerCtaMax, "shared memory");
};

struct BkUnit {
    int r, bb, kvh, n;       // n: row tiles from `first` on that see the block
    int e;                   // fp16: dS is held times 2^e
    int64_t h, kv0, first;
    int64_t len, pos0;
};

struct BkBars {
    uint64_t k_full, v_full, k_empty, v_empty;  // key block landed; its last scores have read it
    uint64_t q_full[4], q_empty[4], g_full[4], g_empty[4];
    uint64_t clean[4];  // rows that see no key zeroed in both tiles
    uint64_t s_full, p_ready, dp_full, ds_ready;
    uint64_t acc_full, acc_free;
    uint64_t drain;
    uint32_t tmem;
    CtaLife life;
    AbUnitBoard<BkUnit> board;
};
static_assert(sizeof(BkBars) <= 1024, "barriers");

template <bool F16>  // called by a whole warp
__device__ __forceinline__ BkUnit bk_unit(const AttnBwdArgs& a, int64_t u)
{
    const AttnShape& s = a.s;
    BkUnit t;
    int64_t block;
    attn_order(a.kv_order, u, &t.h, &block);  // the first keys are seen by the most rows
    t.kv0 = block * kAttnRows;
    ab_head(s, t.h, &t.r, &t.bb, &t.kvh);
    attn_limits(s, t.bb, &t.len, &t.pos0);
    // row i sees key kv0 when i >= kv0 - pos0
    const int64_t row = max(int64_t(0), t.kv0 - t.pos0);
    t.first = row / a.tile_tokens;
    t.n = t.kv0 < t.len && t.first < a.q_tiles ? int(a.q_tiles - t.first) : 0;
    t.e = 0;
    if (F16 && t.n > 0) {
        const float2* rows = a.row_bounds + (t.h * a.q_tiles + t.first) * 2;
        float2 most = make_float2(0.0f, 0.0f);
#pragma unroll 4
        for (int64_t i = threadIdx.x & 31; i < 2 * int64_t(t.n); i += 32) {
            const float2 x = rows[i];
            most = make_float2(fmaxf(most.x, x.x), fmaxf(most.y, x.y));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            most.x = fmaxf(most.x, __shfl_xor_sync(0xffffffffu, most.x, off));
            most.y = fmaxf(most.y, __shfl_xor_sync(0xffffffffu, most.y, off));
        }
        t.e = ab_exponent(most.x * a.key_norms[t.h * a.kv_order.blocks + block] + most.y);
    }
    return t;
}

// Rows at the start of a unit's first tile that see no key at all (a start before the first key): their
// P and dS are zero, but zero times what Q and dO hold there may be NaN. Later tiles have none, and
// tiles with such rows only are not walked.
__device__ __forceinline__ int bk_hidden(const AttnBwdArgs& a, const BkUnit& t)
{
    const int64_t tokens = -t.pos0 - t.first * a.tile_tokens;
    return tokens > 0 ? int(min(tokens, int64_t(a.tile_tokens))) * a.s.group : 0;
}

template <int DP, bool F16>
__global__ void __launch_bounds__(kAbThreads, 1)
    attn_bwd_kv_kernel(const __grid_constant__ AttnBwdArgs a)
{
    using L = BkSmem<DP>;
    using E = ElemT<F16>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    BkBars& bars = *reinterpret_cast<BkBars*>(smem);
    volatile CtaLife* life = &bars.life;
    const AttnShape& s = a.s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (s.d + 15) / 16, halves = (s.d + 63) / 64;
    const int64_t units = a.kv_order.heads * a.kv_order.blocks;
    constexpr int K = L::kStages;

    if (threadIdx.x == 0) {
        mbar_init(&bars.k_full, 1);
        mbar_init(&bars.v_full, 1);
        mbar_init(&bars.k_empty, 1);
        mbar_init(&bars.v_empty, 1);
        for (int k = 0; k < K; ++k) {
            mbar_init(&bars.q_full[k], 1);
            mbar_init(&bars.q_empty[k], s.q_start ? 2 : 1);  // the products, and warp 18
            mbar_init(&bars.g_full[k], 1);
            mbar_init(&bars.g_empty[k], s.q_start ? 2 : 1);
            mbar_init(&bars.clean[k], 1);
        }
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.p_ready, 16);
        mbar_init(&bars.dp_full, 1);
        mbar_init(&bars.ds_ready, 16);
        mbar_init(&bars.acc_full, 1);
        mbar_init(&bars.acc_free, 16);
        ab_board_init(bars.board, s.q_start ? 19 : 18);  // warps 0-17, and 18
        mbar_init(&bars.drain, 1);
        life_init(bars.life, s.wait_us, kAbThreads / 32);
        fence_barrier_init();
    }
    // Rows of a tile past tile_tokens * group never arrive: they are summed over with P = dS = 0,
    // and must be numbers.
    if (a.tile_tokens * s.group < kAttnRows) {
        for (int i = threadIdx.x * 16; i < 2 * K * L::kTile; i += kAbThreads * 16)
            st_shared_v4(smem + L::kQ + i, make_uint4(0, 0, 0, 0));
        fence_proxy_async_shared();
    }
    if (warp == kAbMmaWarp) tmem_alloc(&bars.tmem);
    wait_for_previous();  // the row statistics
    if (threadIdx.x == 0) release_word(a.ready, 1);
    fence_proxy_async_global();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    let_next_start();  // dQ's CTAs fill the SMs that this kernel has no more units for
    const uint32_t tmem = bars.tmem;

    if (warp == kAbLoadWarp) {
        if (lane == 0) {
            StageRing ring;
            uint32_t blocks[2] = {0, 0};    // copies issued: of K and V blocks,
            int64_t q_tiles = 0, g_tiles = 0;  // of q and dO tiles
            const uint32_t q_bytes = uint32_t(halves) * a.tile_tokens * s.group * 128u;
            const uint32_t kv_bytes = uint32_t(halves) * L::kHalf;
            bool ok = true;
            AbUnits<BkUnit> source{&bars.board, life};
            BkUnit t;
            while (ok && source.next<false>(&t)) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (ok && blocks[w] > 0)
                        ok = wait_or_dead(w ? &bars.v_empty : &bars.k_empty, (blocks[w] - 1) & 1,
                                          life);
                    if (!ok) break;
                    uint64_t* bar = w ? &bars.v_full : &bars.k_full;
                    mbar_arrive_expect_tx(bar, kv_bytes);
                    for (int h = 0; h < halves; ++h)
                        tensor_g2s_4d(smem + (w ? L::kV : L::kK) + h * L::kHalf,
                                      w ? &a.vmap[t.r] : &a.kmap[t.r], 64 * h, t.kvh, int(t.kv0),
                                      t.bb, bar);
                    ++blocks[w];
                }
                if (!ok) break;
                for (int i = 0; ok && i < t.n; ++i) {
                    const int64_t tile = t.first + i;
                    if (q_tiles >= K) ok = wait_or_dead(&bars.q_empty[ring.s], ring.phase ^ 1u, life);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars.q_full[ring.s], q_bytes + kAbStats);
                    bulk_g2s(smem + L::kStat + ring.s * kAbStats,
                             a.stats + (t.h * a.q_tiles + tile) * kAbStatArrays<F16> * kAttnRows,
                             kAbStats,
                             &bars.q_full[ring.s]);
                    for (int h = 0; h < halves; ++h)
                        tensor_g2s_4d(smem + L::kQ + ring.s * L::kTile + h * L::kHalf, &a.qmap[t.r],
                                      64 * h, t.kvh * s.group, int(tile * a.tile_tokens), t.bb,
                                      &bars.q_full[ring.s]);
                    ++q_tiles;
                    if (g_tiles >= K) ok = wait_or_dead(&bars.g_empty[ring.s], ring.phase ^ 1u, life);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars.g_full[ring.s], q_bytes);
                    for (int h = 0; h < halves; ++h)
                        tensor_g2s_4d(smem + L::kG + ring.s * L::kTile + h * L::kHalf, &a.gmap[t.r],
                                      64 * h, t.kvh * s.group, int(tile * a.tile_tokens), t.bb,
                                      &bars.g_full[ring.s]);
                    life->loads = uint32_t(++g_tiles);
                    ring.next(K);
                }
            }
            // leave no copy into this CTA's shared memory in flight (a loader that gave up may have
            // issued a K block without its V, a q tile without its dO)
            bool drained = true;
            for (int64_t k = max(int64_t(0), q_tiles - K); k < q_tiles; ++k)
                drained &= mbar_wait_bounded(&bars.q_full[k % K], uint32_t((k / K) & 1));
            for (int64_t k = max(int64_t(0), g_tiles - K); k < g_tiles; ++k)
                drained &= mbar_wait_bounded(&bars.g_full[k % K], uint32_t((k / K) & 1));
            if (blocks[0] > 0) drained &= mbar_wait_bounded(&bars.k_full, (blocks[0] - 1) & 1);
            if (blocks[1] > 0) drained &= mbar_wait_bounded(&bars.v_full, (blocks[1] - 1) & 1);
            if (!drained) atomicOr(&g_attn_bwd_status, kStatusDrainTimeout);
        }
        __syncwarp();
    } else if (warp == kAbMmaWarp) {
        if (elect_one()) {
            const uint32_t id_s = tc_idesc(F16, kAttnRows, false);
            const uint32_t id_d = tc_idesc(F16, 16 * nk, true);
            const uint64_t k_desc = tc_desc_k(smem_u32(smem + L::kK));
            const uint64_t v_desc = tc_desc_k(smem_u32(smem + L::kV));
            const uint64_t q_desc = tc_desc_k(smem_u32(smem + L::kQ));
            const uint64_t g_desc = tc_desc_k(smem_u32(smem + L::kG));
            const uint64_t qt_desc = tc_desc_mn(smem_u32(smem + L::kQ), L::kHalf);
            const uint64_t gt_desc = tc_desc_mn(smem_u32(smem + L::kG), L::kHalf);
            StageRing ring;
            uint32_t uses = 0, tiles = 0;
            uint32_t cleaned = 0;  // parity of each stage's `clean`
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return ok = ok && wait_or_dead(bar, parity, life);
            };
            auto scores = [&](uint32_t d, uint64_t key, uint64_t row, uint64_t* bar) {
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    if (ks >= nk) break;
                    const uint32_t off = ((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4;
                    tc_mma_ss(tmem + d, key + off, row + off, id_s, ks > 0);
                }
                tc_commit(bar);
            };
            auto sums = [&](uint32_t d, uint32_t p, uint64_t row, bool first) {
#pragma unroll
                for (int ks = 0; ks < kAttnRows / 16; ++ks)  // each warpgroup's 32 columns in 16
                    tc_mma_ts(tmem + d, tmem + p + (ks >> 1) * 32 + (ks & 1) * 8,
                              row + ks * (2048 >> 4), id_d, !first || ks > 0);
            };
            // S^T (dP^T) of the ring's next row tile; `first`, `last` of unit u
            auto next_s = [&](bool first, bool last, uint32_t use, const BkUnit& u) {
                if (first) wait(&bars.k_full, use & 1);
                if (!wait(&bars.q_full[ring.s], ring.phase)) return;
                if (first && s.q_start && bk_hidden(a, u) > 0) {
                    if (!wait(&bars.clean[ring.s], (cleaned >> ring.s) & 1)) return;
                    cleaned ^= 1u << ring.s;
                }
                tc_fence_after();
                scores(kBkS, k_desc, q_desc + ring.s * (L::kTile >> 4), &bars.s_full);
                if (last) tc_commit(&bars.k_empty);
            };
            auto next_dp = [&](bool first, bool last, uint32_t use) {
                if (first) wait(&bars.v_full, use & 1);
                if (!wait(&bars.g_full[ring.s], ring.phase)) return;
                tc_fence_after();
                scores(kBkDp, v_desc, g_desc + ring.s * (L::kTile >> 4), &bars.dp_full);
                if (last) tc_commit(&bars.v_empty);
            };
            AbUnits<BkUnit> source{&bars.board, life};
            BkUnit t, next;
            bool live = source.next<false>(&t);
            if (live) {
                next_s(true, t.n == 1, 0, t);
                next_dp(true, t.n == 1, 0);
            }
            while (live && ok) {
                bool more = false;
                for (int i = 0; ok && i < t.n; ++i, ++tiles) {
                    const int at = ring.s;
                    const bool end = i + 1 == t.n;           // the next tile is the next unit's
                    if (end) more = source.next<false>(&next);
                    const bool last = end ? next.n == 1 : i + 2 == t.n;
                    ring.next(K);
                    wait(&bars.p_ready, tiles & 1);
                    if (i == 0 && uses > 0) wait(&bars.acc_free, (uses - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    sums(kBkDv, kBkS, gt_desc + at * (L::kTile >> 4), i == 0);
                    tc_commit(&bars.g_empty[at]);
                    if (!end || more) next_s(end, last, uses + 1, next);
                    if (!wait(&bars.ds_ready, tiles & 1)) break;
                    tc_fence_after();
                    sums(kBkDk, kBkDp, qt_desc + at * (L::kTile >> 4), i == 0);
                    tc_commit(&bars.q_empty[at]);
                    if (end) tc_commit(&bars.acc_full);
                    if (!end || more) next_dp(end, last, uses + 1);
                }
                ++uses;
                t = next;
                live = more;
            }
            tc_commit(&bars.drain);  // every product complete before tensor memory is given back
            if (!mbar_wait_bounded(&bars.drain, 0)) atomicOr(&g_attn_bwd_status, kStatusDrainTimeout);
        }
        __syncwarp();
    } else if (warp == kAbCleanWarp) {
        if (s.q_start) {
            StageRing ring;
            AbUnits<BkUnit> source{&bars.board, life};
            BkUnit t;
            bool ok = true;
            while (ok && source.next<true>(&t)) {
                for (int i = 0; ok && i < t.n; ++i) {
                    ok = __all_sync(0xffffffffu, wait_or_dead(&bars.q_full[ring.s], ring.phase, life));
                    ok = ok &&
                         __all_sync(0xffffffffu, wait_or_dead(&bars.g_full[ring.s], ring.phase, life));
                    if (!ok) break;
                    const int hidden = i == 0 ? bk_hidden(a, t) : 0;
                    if (hidden > 0) {
                        for (int h = 0; h < halves; ++h)
                            for (int w = lane; w < hidden * 8; w += 32) {
                                const int at = ring.s * L::kTile + h * L::kHalf + w * 16;
                                st_shared_v4(smem + L::kQ + at, make_uint4(0, 0, 0, 0));
                                st_shared_v4(smem + L::kG + at, make_uint4(0, 0, 0, 0));
                            }
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.clean[ring.s]);
                    }
                    // every stage waits for this warp, so that it neither runs ahead of the ring
                    // nor falls a turn behind
                    if (lane == 0) {
                        mbar_arrive(&bars.q_empty[ring.s]);
                        mbar_arrive(&bars.g_empty[ring.s]);
                    }
                    ring.next(K);
                }
            }
        }
        __syncwarp();
    } else if (warp == kAbUnitWarp) {
        ab_publish<BkUnit>(
            bars.board, units, life, [&](int64_t u) { return bk_unit<F16>(a, u); },
            [&](const BkUnit& t) {  // keys that no row sees
                for (int i = lane; i < 2 * kAttnRows; i += 32) {
                    const int64_t key = t.kv0 + i % kAttnRows;
                    if (key >= s.Skv) continue;
                    uint8_t* out = (i >= kAttnRows ? a.dv[t.r] : a.dk[t.r]) +
                                   ((int64_t(t.bb) * s.Skv + key) * s.m[t.r] + t.kvh) * s.d * 2;
                    for (int c = 0; c < s.d * 2; c += 16) st_v4(out + c, make_uint4(0, 0, 0, 0));
                }
            });
    } else if (warp < kAbLoadWarp) {
        const int wg = warp >> 2;  // columns 32 wg .. 32 wg + 31; then a half of dK (0, 1) or dV
        const int row = threadIdx.x & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;
        const uint32_t s_at = tmem + lanes + kBkS + wg * 32;
        const uint32_t dp_at = tmem + lanes + kBkDp + wg * 32;
        const float sl2 = s.scale * 1.4426950408889634f;
        StageRing ring;
        uint32_t uses = 0, tiles = 0;
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
        AbUnits<BkUnit> source{&bars.board, life};
        BkUnit t;
        while (ok && source.next<true>(&t)) {
            const int64_t key = t.kv0 + row;
            // columns of the unit's first tile that see this key begin here, of each next one
            // tile_tokens * group columns earlier
            int64_t lo = (key - t.pos0 - t.first * a.tile_tokens) * s.group - 32 * wg;
            if (key >= t.len) lo = int64_t(1) << 40;
            const float2 ds2 = make_float2(ab_power(t.e - kAttnPBits), ab_power(t.e - kAttnPBits));
            for (int i = 0; i < t.n; ++i, lo -= a.tile_tokens * s.group) {
                const int from = int(max(int64_t(-1), min(lo, int64_t(32))));
                ok = all(&bars.q_full[ring.s], ring.phase);  // the tile's lse and D
                ok = ok && all(&bars.s_full, tiles & 1);
                if (!ok) break;
                tc_fence_after();
                const float4* z4 =
                    reinterpret_cast<const float4*>(smem + L::kStat + ring.s * kAbStats) + wg * 8;
                uint32_t x[32];
                tmem_ld32(s_at, x);
                tmem_wait_ld(x);
                const float2 k2 = make_float2(sl2, sl2);
                uint32_t p[16];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 z = z4[c];
                    const float2 e = __ffma2_rn(make_float2(__uint_as_float(x[4 * c]),
                                                            __uint_as_float(x[4 * c + 1])),
                                                k2, make_float2(-z.x, -z.y));
                    const float2 f = __ffma2_rn(make_float2(__uint_as_float(x[4 * c + 2]),
                                                            __uint_as_float(x[4 * c + 3])),
                                                k2, make_float2(-z.z, -z.w));
                    x[4 * c] = __float_as_uint(ex2(e.x));
                    x[4 * c + 1] = __float_as_uint(ex2(e.y));
                    x[4 * c + 2] = __float_as_uint(ex2(f.x));
                    x[4 * c + 3] = __float_as_uint(ex2(f.y));
                }
                const bool masked = __any_sync(0xffffffffu, from > 0);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c < from) x[c] = 0;
                }
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    p[c] = E::pack(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
                tmem_st16(s_at, p);
                arrive(&bars.p_ready);

                ok = all(&bars.dp_full, tiles & 1);
                if (!ok) break;
                tc_fence_after();
                const float4* d4 = z4 + kAttnRows / 4;
                uint32_t y[32];
                tmem_ld32(dp_at, y);
                tmem_wait_ld(y);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 dd = d4[c];
                    float2 v = ab_ds(x[4 * c], x[4 * c + 1], y[4 * c], y[4 * c + 1],
                                     make_float2(-dd.x, -dd.y));
                    float2 w = ab_ds(x[4 * c + 2], x[4 * c + 3], y[4 * c + 2], y[4 * c + 3],
                                     make_float2(-dd.z, -dd.w));
                    if (F16) {
                        v = __fmul2_rn(v, ds2);
                        w = __fmul2_rn(w, ds2);
                    }
                    p[2 * c] = E::pack(v.x, v.y);
                    p[2 * c + 1] = E::pack(w.x, w.y);
                }
                if (masked) {  // zero times what lies past the last key may be NaN
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if (2 * c < from) p[c] &= 0xFFFF0000u;
                        if (2 * c + 1 < from) p[c] &= 0x0000FFFFu;
                    }
                }
                tmem_st16(dp_at, p);
                arrive(&bars.ds_ready);
                ++tiles;
                ring.next(K);
            }
            if (!ok) break;
            ok = all(&bars.acc_full, uses & 1);
            if (!ok) break;
            tc_fence_after();
            uint8_t* out = (wg >= 2 ? a.dv[t.r] : a.dk[t.r]) +
                           ((int64_t(t.bb) * s.Skv + key) * s.m[t.r] + t.kvh) * s.d * 2;
            const float f = wg >= 2 ? (F16 ? ab_power(-kAttnPBits) : 1.0f)
                                    : (F16 ? s.scale * ab_power(-t.e) : s.scale);
            constexpr int kCols = DP / 2;
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) {
                const int col = (wg & 1) * kCols + c * 32;
                uint32_t y[32];
                tmem_ld32(tmem + lanes + (wg >= 2 ? kBkDv : kBkDk) + col, y);
                tmem_wait_ld(y);
                if (c == kCols / 32 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.acc_free);
                }
                if (key < s.Skv) ab_store<E>(out, col, s.d, y, f);
            }
            ++uses;
        }
    }
    life_end(bars.life, warp == kAbUnitWarp);
    __syncthreads();
    if (threadIdx.x == 0 && life_status(bars.life) != 0)
        atomicOr(&g_attn_bwd_status, life_status(bars.life));
    if (warp == kAbMmaWarp) tmem_free(tmem);
}

// ---- dQ -----------------------------------------------------------------------------------------

// Tensor memory columns: Q (16 bits, two a column), dS (the same), S, dP, dQ. Lanes are rows of q,
// columns keys.
constexpr int kBqQ = 0, kBqDs = 64, kBqS = 128, kBqDp = 256, kBqDq = 384;

template <int DP>
struct BqSmem {
    static constexpr int kTile = kAttnRows * DP * 2;
    static constexpr int kHalf = kAttnRows * 128;
    static constexpr int kStages = DP == 128 ? 6 : 8;
    static constexpr int kG = 1024;          // dO, the unit's
    static constexpr int kRing = kG + kTile;  // Q K0 V0 K1 V1 ... of each unit
    static constexpr int kTotal = kRing + kStages * kTile;
    static_assert(kTotal + 1024 <= kSmemPerCtaMax, "shared memory");
};

struct BqUnit {
    int r, bb, kvh, n;  // n: key blocks that the tile sees
    float norm;         // fp16: the largest |v| in them
    int64_t h, tile, tok0, len, pos0;
};

struct BqBars {
    uint64_t full[8], empty[8], clean[8];  // ring stages; clean: K rows past the last key zeroed
    uint64_t g_full, g_empty;              // dO landed; its last scores have read it
    uint64_t q_ready;                      // Q in tensor memory
    uint64_t s_full, s_read, dp_full, dp_read;  // scores complete; read
    uint64_t ds_ready, dq_done;            // dS written; summed up
    uint64_t acc_full, acc_free, drain;
    uint32_t tmem;
    int seen;
    CtaLife life;
    AbUnitBoard<BqUnit> board;
};
static_assert(sizeof(BqBars) <= 1024, "barriers");

template <bool F16>  // called by a whole warp
__device__ __forceinline__ BqUnit bq_unit(const AttnBwdArgs& a, int64_t u)
{
    const AttnShape& s = a.s;
    BqUnit t;
    attn_order(a.q_order, u, &t.h, &t.tile);
    if (s.causal) t.tile = a.q_tiles - 1 - t.tile;  // the longest rows first
    t.tok0 = t.tile * a.tile_tokens;
    ab_head(s, t.h, &t.r, &t.bb, &t.kvh);
    attn_limits(s, t.bb, &t.len, &t.pos0);
    const int64_t last = min(t.tok0 + a.tile_tokens, s.Sq) - 1;
    const int64_t keys = max(int64_t(0), min(t.len, t.pos0 + last + 1));
    t.n = int((keys + kAttnRows - 1) / kAttnRows);
    t.norm = 0.0f;
    if (F16) {
        const float* norms = a.key_norms + t.h * a.kv_order.blocks;
#pragma unroll 4
        for (int i = threadIdx.x & 31; i < t.n; i += 32) t.norm = fmaxf(t.norm, norms[i]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            t.norm = fmaxf(t.norm, __shfl_xor_sync(0xffffffffu, t.norm, off));
    }
    return t;
}

// Rows of a key block past the batch element's last key that the tensor holds; kAttnRows: none.
__device__ __forceinline__ int bq_past(const AttnShape& s, const BqUnit& t, int block)
{
    const int64_t past = t.len - int64_t(block) * kAttnRows;
    return past >= kAttnRows || t.len >= s.Skv ? kAttnRows : int(past);
}

// Q goes to tensor memory (the S products then read half as much shared memory), S and dP are free
// again as soon as the threads have read them, and dS has columns of its own, so that the products
// run S, dP of the next block and dQ of this one without waiting for the threads' arithmetic.
template <int DP, bool F16>
__global__ void __launch_bounds__(kAbThreads, 1)
    attn_bwd_q_kernel(const __grid_constant__ AttnBwdArgs a)
{
    using L = BqSmem<DP>;
    using E = ElemT<F16>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    BqBars& bars = *reinterpret_cast<BqBars*>(smem);
    volatile CtaLife* life = &bars.life;
    const AttnShape& s = a.s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (s.d + 15) / 16, halves = (s.d + 63) / 64;
    const int64_t units = a.q_order.heads * a.q_order.blocks;
    constexpr int K = L::kStages;

    if (threadIdx.x == 0) {
        for (int k = 0; k < K; ++k) {
            mbar_init(&bars.full[k], 1);
            mbar_init(&bars.empty[k], s.ragged ? 2 : 1);  // the products, and warp 18
            mbar_init(&bars.clean[k], 1);
        }
        mbar_init(&bars.g_full, 1);
        mbar_init(&bars.g_empty, 1);
        mbar_init(&bars.q_ready, 16);
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.s_read, 16);
        mbar_init(&bars.dp_full, 1);
        mbar_init(&bars.dp_read, 16);
        mbar_init(&bars.ds_ready, 16);
        mbar_init(&bars.dq_done, 1);
        mbar_init(&bars.acc_full, 1);
        mbar_init(&bars.acc_free, 16);
        ab_board_init(bars.board, s.ragged ? 19 : 18);  // warps 0-17, and 18
        mbar_init(&bars.drain, 1);
        life_init(bars.life, s.wait_us, kAbThreads / 32);
        // The kernel in front (dK, dV) waited for the statistics before it let this one start. What it
        // had seen then is seen here through `ready`; if that is not there yet, after its end.
        bars.seen = acquire_word(a.ready) == 1;
        fence_barrier_init();
    }
    if (warp == kAbMmaWarp) tmem_alloc(&bars.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!bars.seen) wait_for_previous();
    fence_proxy_async_global();
    const uint32_t tmem = bars.tmem;

    if (warp == kAbLoadWarp) {
        if (lane == 0) {
            StageRing ring;
            uint32_t uses = 0;
            int64_t issued = 0;
            const uint32_t q_bytes = uint32_t(halves) * a.tile_tokens * s.group * 128u;
            const uint32_t kv_bytes = uint32_t(halves) * L::kHalf;
            bool ok = true;
            auto stage = [&](const CUtensorMap* map, uint32_t bytes, int head, int row, int bb) {
                if (issued >= K) ok = wait_or_dead(&bars.empty[ring.s], ring.phase ^ 1u, life);
                if (!ok) return;
                mbar_arrive_expect_tx(&bars.full[ring.s], bytes);
                for (int h = 0; h < halves; ++h)
                    tensor_g2s_4d(smem + L::kRing + ring.s * L::kTile + h * L::kHalf, map, 64 * h,
                                  head, row, bb, &bars.full[ring.s]);
                life->loads = uint32_t(++issued);
                ring.next(K);
            };
            AbUnits<BqUnit> source{&bars.board, life};
            BqUnit t;
            while (ok && source.next<false>(&t)) {
                stage(&a.qmap[t.r], q_bytes, t.kvh * s.group, int(t.tok0), t.bb);
                if (ok) stage(&a.kmap[t.r], kv_bytes, t.kvh, 0, t.bb);
                if (ok && uses > 0) ok = wait_or_dead(&bars.g_empty, (uses - 1) & 1, life);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars.g_full, q_bytes);
                for (int h = 0; h < halves; ++h)
                    tensor_g2s_4d(smem + L::kG + h * L::kHalf, &a.gmap[t.r], 64 * h,
                                  t.kvh * s.group, int(t.tok0), t.bb, &bars.g_full);
                ++uses;
                for (int j = 1; ok && j < 2 * t.n; ++j)
                    stage((j & 1) ? &a.vmap[t.r] : &a.kmap[t.r], kv_bytes, t.kvh,
                          (j >> 1) * kAttnRows, t.bb);
            }
            bool drained = true;  // leave no copy into this CTA's shared memory in flight
            for (int64_t k = max(int64_t(0), issued - K); k < issued; ++k)
                drained &= mbar_wait_bounded(&bars.full[k % K], uint32_t((k / K) & 1));
            if (uses > 0) drained &= mbar_wait_bounded(&bars.g_full, (uses - 1) & 1);
            if (!drained) atomicOr(&g_attn_bwd_status, kStatusDrainTimeout);
        }
        __syncwarp();
    } else if (warp == kAbCleanWarp) {
        // dS is zero past the last key, but zero times what K holds there may be NaN
        if (s.ragged) {
            StageRing ring;
            AbUnits<BqUnit> source{&bars.board, life};
            BqUnit t;
            bool ok = true;
            while (ok && source.next<true>(&t)) {
                for (int j = -1; ok && j < 2 * t.n; ++j) {  // Q K0 V0 K1 V1 ...
                    ok = __all_sync(0xffffffffu, wait_or_dead(&bars.full[ring.s], ring.phase, life));
                    if (!ok) break;
                    const int past = j < 0 || (j & 1) ? kAttnRows : bq_past(s, t, j >> 1);
                    if (past < kAttnRows) {
                        for (int h = 0; h < halves; ++h)
                            for (int w = past * 8 + lane; w < kAttnRows * 8; w += 32)
                                st_shared_v4(smem + L::kRing + ring.s * L::kTile + h * L::kHalf +
                                                 w * 16,
                                             make_uint4(0, 0, 0, 0));
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.clean[ring.s]);
                    }
                    // every stage waits for this warp, so that it neither runs ahead of the ring
                    // nor falls a turn behind
                    if (lane == 0) mbar_arrive(&bars.empty[ring.s]);
                    ring.next(K);
                }
            }
        }
        __syncwarp();
    } else if (warp == kAbMmaWarp) {
        if (elect_one()) {
            const uint32_t id_s = tc_idesc(F16, kAttnRows, false);
            const uint32_t id_d = tc_idesc(F16, 16 * nk, true);
            const uint64_t g_desc = tc_desc_k(smem_u32(smem + L::kG));
            const uint64_t kv_desc = tc_desc_k(smem_u32(smem + L::kRing));
            const uint64_t kt_desc = tc_desc_mn(smem_u32(smem + L::kRing), L::kHalf);
            StageRing ring;
            uint32_t uses = 0, blocks = 0;
            uint32_t cleaned = 0;  // parity of each stage's `clean`
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return ok = ok && wait_or_dead(bar, parity, life);
            };
            // S of the ring's next block, whose stage it returns; dP of the V in the stage after it.
            // `first` of unit number `use`: its queries come before its keys.
            auto make_s = [&](bool first, uint32_t use) {
                if (first) {
                    if (!wait(&bars.q_ready, use & 1)) return 0;
                    mbar_arrive(&bars.empty[ring.s]);
                    ring.next(K);
                }
                const int stage = ring.s;
                if (!wait(&bars.full[stage], ring.phase)) return stage;
                tc_fence_after();
                const uint64_t key = kv_desc + stage * (L::kTile >> 4);
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    if (ks >= nk) break;
                    tc_mma_ts(tmem + kBqS, tmem + kBqQ + ks * 8,
                              key + (((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4), id_s, ks > 0);
                }
                tc_commit(&bars.s_full);
                ring.next(K);
                return stage;
            };
            auto make_dp = [&](bool first, bool last, uint32_t use) {
                if (first) wait(&bars.g_full, use & 1);
                if (!wait(&bars.full[ring.s], ring.phase)) return;
                tc_fence_after();
                const uint64_t key = kv_desc + ring.s * (L::kTile >> 4);
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    if (ks >= nk) break;
                    const uint32_t off = ((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4;
                    tc_mma_ss(tmem + kBqDp, g_desc + off, key + off, id_s, ks > 0);
                }
                tc_commit(&bars.dp_full);
                tc_commit(&bars.empty[ring.s]);
                if (last) tc_commit(&bars.g_empty);
                ring.next(K);
            };
            AbUnits<BqUnit> source{&bars.board, life};
            BqUnit t, next;
            bool live = source.next<false>(&t);
            int ks = 0;  // the stage of the current block's K
            if (live) {
                ks = make_s(true, 0);
                make_dp(true, t.n == 1, 0);
            }
            while (live && ok) {
                bool more = false;
                for (int j = 0; ok && j < t.n; ++j, ++blocks) {
                    const bool end = j + 1 == t.n;  // the next block is the next unit's
                    if (end) more = source.next<false>(&next);
                    int after = ks;
                    wait(&bars.s_read, blocks & 1);
                    if (!end) after = make_s(false, uses);
                    wait(&bars.dp_read, blocks & 1);
                    if (!end) make_dp(false, j + 2 == t.n, uses);
                    if (s.ragged && bq_past(s, t, j) < kAttnRows) {
                        wait(&bars.clean[ks], (cleaned >> ks) & 1);
                        cleaned ^= 1u << ks;
                    }
                    wait(&bars.ds_ready, blocks & 1);
                    if (j == 0 && uses > 0) wait(&bars.acc_free, (uses - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t kd = kt_desc + ks * (L::kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < kAttnRows / 16; ++kk)
                        tc_mma_ts(tmem + kBqDq, tmem + kBqDs + kk * 8, kd + kk * (2048 >> 4), id_d,
                                  j > 0 || kk > 0);
                    tc_commit(&bars.empty[ks]);
                    tc_commit(&bars.dq_done);
                    if (end) {
                        tc_commit(&bars.acc_full);
                        if (more) {
                            after = make_s(true, uses + 1);
                            make_dp(true, next.n == 1, uses + 1);
                        }
                    }
                    ks = after;
                }
                ++uses;
                t = next;
                live = more;
            }
            tc_commit(&bars.drain);
            if (!mbar_wait_bounded(&bars.drain, 0)) atomicOr(&g_attn_bwd_status, kStatusDrainTimeout);
        }
        __syncwarp();
    } else if (warp == kAbUnitWarp) {
        ab_publish<BqUnit>(
            bars.board, units, life, [&](int64_t u) { return bq_unit<F16>(a, u); },
            [&](const BqUnit& t) {  // rows that see no key
                for (int i = lane; i < kAttnRows; i += 32) {
                    const int tok_in = i / s.group;
                    const int64_t tok = t.tok0 + tok_in;
                    if (tok_in >= a.tile_tokens || tok >= s.Sq) continue;
                    uint8_t* out = a.dq[t.r] + ((int64_t(t.bb) * s.Sq + tok) * s.n[t.r] +
                                                t.kvh * s.group + i - tok_in * s.group) * s.d * 2;
                    for (int c = 0; c < s.d * 2; c += 16) st_v4(out + c, make_uint4(0, 0, 0, 0));
                }
            });
    } else {
        const int wg = warp >> 2;  // keys 32 wg .. 32 wg + 31 of a block; then a quarter of dQ
        const int row = threadIdx.x & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;
        const uint32_t s_at = tmem + lanes + kBqS + wg * 32;
        const uint32_t dp_at = tmem + lanes + kBqDp + wg * 32;
        const uint32_t ds_at = tmem + lanes + kBqDs + wg * 16;
        const float sl2 = s.scale * 1.4426950408889634f;
        const int tok_in = row / s.group, head_in = row - tok_in * s.group;
        uint32_t uses = 0, blocks = 0;
        int64_t stages = 0;  // of the ring before the current unit
        bool ok = true;
        auto all = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_or_dead(bar, parity, life));
        };
        auto arrive = [&](uint64_t* bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // This row of a unit's Q (warpgroups 0, 1: its halves) from its stage to tensor memory, which
        // the scores made so far are done with.
        auto copy = [&](int64_t at) {
            const int stage = int(at % K);
            ok = all(&bars.full[stage], uint32_t(at / K) & 1);
            if (!ok) return;
            if (wg < halves) {
                const uint8_t* from = smem + L::kRing + stage * L::kTile + wg * L::kHalf + row * 128;
                uint32_t v[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 w = ld_shared_v4(from + ((c ^ (row & 7)) << 4));
                    v[4 * c] = w.x, v[4 * c + 1] = w.y, v[4 * c + 2] = w.z, v[4 * c + 3] = w.w;
                }
                tmem_st32(tmem + lanes + kBqQ + wg * 32, v);
                tmem_wait_st();
            }
            arrive(&bars.q_ready);
        };
        AbUnits<BqUnit> source{&bars.board, life};
        BqUnit t, next;
        bool live = source.next<true>(&t);
        if (live) copy(0);
        while (live && ok) {
            const int64_t tok = t.tok0 + tok_in;
            const bool valid = tok_in < a.tile_tokens && tok < s.Sq;
            const float* stat =
                a.stats + (t.h * a.q_tiles + t.tile) * kAbStatArrays<F16> * kAttnRows + row;
            float z = -stat[0], f = s.scale;
            const float delta = stat[kAttnRows];
            if (F16) {
                const int e = ab_exponent(fmaf(stat[2 * kAttnRows], t.norm, fabsf(delta)));
                z += float(e - kAttnPBits);
                f *= ab_power(-e);
            }
            int64_t left = min(t.len, t.pos0 + tok + 1) - 32 * wg;  // visible keys from here on
            for (int j = 0; j < t.n; ++j, ++blocks, left -= kAttnRows) {
                const int seen = int(max(int64_t(0), min(left, int64_t(32))));
                ok = all(&bars.s_full, blocks & 1);
                if (!ok) break;
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32(s_at, x);
                tmem_wait_ld(x);
                arrive(&bars.s_read);
                const float2 k2 = make_float2(sl2, sl2), z2 = make_float2(z, z);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float2 e = __ffma2_rn(
                        make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), k2, z2);
                    x[2 * c] = __float_as_uint(ex2(e.x));
                    x[2 * c + 1] = __float_as_uint(ex2(e.y));
                }
                const bool masked = __any_sync(0xffffffffu, seen < 32);
                ok = all(&bars.dp_full, blocks & 1);
                if (!ok) break;
                tc_fence_after();
                uint32_t y[32], p[16];
                tmem_ld32(dp_at, y);
                tmem_wait_ld(y);
                arrive(&bars.dp_read);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float2 v = ab_ds(x[2 * c], x[2 * c + 1], y[2 * c], y[2 * c + 1],
                                           make_float2(-delta, -delta));
                    p[c] = E::pack(v.x, v.y);
                }
                if (masked) {  // zero times what lies past the last key may be NaN
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if (2 * c >= seen) p[c] &= 0xFFFF0000u;
                        if (2 * c + 1 >= seen) p[c] &= 0x0000FFFFu;
                    }
                }
                if (blocks > 0) ok = all(&bars.dq_done, (blocks - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                tmem_st16(ds_at, p);
                tmem_wait_st();
                arrive(&bars.ds_ready);
                if (j + 1 == t.n) {  // the next unit's queries (its S then runs beside the last dQ)
                    stages += 1 + 2 * t.n;
                    live = source.next<true>(&next);
                    if (live) copy(stages);
                    if (!ok) break;
                }
            }
            if (!ok) break;
            ok = all(&bars.acc_full, uses & 1);
            if (!ok) break;
            tc_fence_after();
            uint8_t* out = a.dq[t.r] + ((int64_t(t.bb) * s.Sq + tok) * s.n[t.r] +
                                        t.kvh * s.group + head_in) * s.d * 2;
            constexpr int kCols = DP / 4;
            uint32_t y[kCols];
            if constexpr (kCols == 32)
                tmem_ld32(tmem + lanes + kBqDq + wg * kCols, y);
            else
                tmem_ld16(tmem + lanes + kBqDq + wg * kCols, y);
            tmem_wait_ld(y);
            arrive(&bars.acc_free);
            if (valid) ab_store<E>(out, wg * kCols, s.d, y, f);
            ++uses;
            t = next;
        }
    }
    life_end(bars.life, warp == kAbUnitWarp);
    wait_for_previous();  // dK and dV are done when this kernel is (nothing here reads them)
    __syncthreads();
    if (threadIdx.x == 0 && life_status(bars.life) != 0)
        atomicOr(&g_attn_bwd_status, life_status(bars.life));
    if (warp == kAbMmaWarp) tmem_free(tmem);
}

template <int DP, bool F16>
static cudaError_t ab_launch(const AttnBwdArgs& a, cudaStream_t stream, int device, int64_t cap,
                             int sm_count)
{
    static std::atomic<unsigned long long> raised{0};
    const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0;
    constexpr int smem_kv = BkSmem<DP>::kTotal + 1024, smem_q = BqSmem<DP>::kTotal + 1024;
    cudaError_t e;
    if (bit && !(raised.load() & bit)) {
        e = cudaFuncSetAttribute(attn_bwd_kv_kernel<DP, F16>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem_kv);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(attn_bwd_q_kernel<DP, F16>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem_q);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit);
    }
    const int64_t heads = a.q_order.heads;
    const int64_t parts = 2 * heads * a.q_tiles + (F16 ? heads * a.kv_order.blocks : 0);
    const bool early = cap == kAttnMostCtas;  // (two at a time together would pass a cap)
    attn_bwd_stats_kernel<F16, DP / 8><<<unsigned(parts < cap ? parts : cap), 256, 0, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = attn_launch_early(attn_bwd_kv_kernel<DP, F16>,
                          attn_ctas(heads * a.kv_order.blocks, cap, sm_count), kAbThreads, smem_kv,
                          stream, a, early);
    if (e != cudaSuccess) return e;
    return attn_launch_early(attn_bwd_q_kernel<DP, F16>, attn_ctas(heads * a.q_tiles, cap, sm_count),
                             kAbThreads, smem_q, stream, a, early);
}

// The three launches over all ranks. The shape, every pointer and the workspace are set in `a`.
cudaError_t attn_bwd_launch(AttnBwdArgs& a, const void* const* q, const void* const* k,
                            const void* const* v, cudaStream_t stream, int device, int64_t cap,
                            int sm_count)
{
    const AttnShape& s = a.s;
    if (s.head_begin[s.W] == 0) return cudaSuccess;
    for (int r = 0; r < s.W; ++r) {
        if (s.n[r] == 0) continue;
        auto rows = [&](CUtensorMap* map, const void* p) {
            return encode_head_map(map, p, s.f16, s.d, s.n[r], s.Sq, s.b, s.group, a.tile_tokens);
        };
        auto keys = [&](CUtensorMap* map, const void* p) {
            return encode_head_map(map, p, s.f16, s.d, s.m[r], s.Skv, s.b, 1, kAttnRows);
        };
        if (!rows(&a.qmap[r], q[r]) || !rows(&a.gmap[r], a.go[r]) || !keys(&a.kmap[r], k[r]) ||
            !keys(&a.vmap[r], v[r]))
            return cudaErrorInvalidValue;
    }
    if (s.d <= 64)
        return s.f16 ? ab_launch<64, true>(a, stream, device, cap, sm_count)
                     : ab_launch<64, false>(a, stream, device, cap, sm_count);
    return s.f16 ? ab_launch<128, true>(a, stream, device, cap, sm_count)
                 : ab_launch<128, false>(a, stream, device, cap, sm_count);
}

cudaError_t attn_bwd_status(unsigned* status, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_attn_bwd_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_bwd_status, &zero, sizeof(unsigned));
}

}  // namespace uly
