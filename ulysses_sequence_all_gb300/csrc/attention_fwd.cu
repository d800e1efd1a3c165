// attention_fwd.cu -- attention of every rank's heads over the whole sequence, between the two
// relayouts (fast-ulysses 0.2.1, README, "Quick start": the attention of a sequence-parallel block
// runs on the head shards that mode 0 delivers).
//
// Per query row i of a head, over the keys j that it sees (j below the batch element's key count
// and, causal, j <= position of i): o_i = sum_j exp(s_ij - m_i) v_j / l_i, s_ij = scale q_i . k_j,
// m_i = max_j s_ij, l_i = sum_j exp(s_ij - m_i), and lse_i = m_i + log l_i. A row that sees no key
// gives zeros and lse = -infinity.
//
// One pass over the keys in blocks of 128 with the running maximum and sum: 4 d flops per (row,
// key) on the tensor cores, one exponential. The kernel is bound by the tensor cores where d = 128
// and by exponentials and products alike where d = 64; with few rows by reading the keys.
//
// A CTA (one per SM, 352 threads) takes two tiles of 128 query rows that share their keys. Warp 8
// loads (tensor maps, swizzled): the query tiles, then a ring of key and value blocks. Warp 9
// issues the products: S = Q K^T of one tile while the other tile's 128 threads turn their S into
// probabilities, so the tensor cores always have one tile's work. Warps 0-3 and 4-7 are the two
// tiles' softmax: tensor memory gives a thread a whole row, so maximum and sum need no exchange.
// P goes back to tensor memory over its own S in 16 bits, rounded to nearest (unit-scale values
// in an fp32 sum: the output itself is rounded to the same type), and is the A operand of O += P V
// there. O stays in tensor memory; it is rescaled only when a row's maximum has grown by more than
// 2^8 since its last scale (P then stays below 2^8, far inside either type), by the softmax threads
// themselves: the block's S is complete only after the previous O product. Warp 10 stores finished
// output tiles, staged in the query tile's place.
//
// With too few tiles to fill the SMs the keys are split into parts, each with its own normalised
// fp32 output and lse, and attn_join_kernel adds them weighted by exp(lse_part - lse).
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

constexpr int kAfThreads = 352;
constexpr int kAfLoadWarp = 8, kAfMmaWarp = 9, kAfStoreWarp = 10;
constexpr float kAfRescale = 8.0f;  // log2 of the growth of a row's maximum that forces a rescale

// Tensor memory columns: the two tiles' scores (their probabilities over them), their outputs.
constexpr int kAfS = 0, kAfO = 256;

template <int DP>
struct AfSmem {
    static constexpr int kTile = kAttnRows * DP * 2;  // a tile of 128 rows; a block of 128 keys
    static constexpr int kHalf = kAttnRows * 128;     // its part of 64 columns
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr int kBars = 0;
    static constexpr int kQ = 1024;
    static constexpr int kRing = kQ + 2 * kTile;
    static constexpr int kTotal = kRing + kStages * kTile;
    static_assert(kTotal + 1024 <= kSmemPerCtaMax, "shared memory");  // and room to align the base
};

struct AfBars {
    uint64_t q_full[2], q_empty[2];   // a tile's queries landed; its output store has read them
    uint64_t s_full[2], p_ready[2];   // scores complete; probabilities (and a rescaled O) written
    uint64_t o_full[2], o_free[2];    // output complete; read out
    uint64_t o_staged[2];             // output tile in shared memory
    uint64_t kv_full[8], kv_empty[8];
    uint64_t drain;
    uint32_t tmem;
    int dead;
};
static_assert(sizeof(AfBars) <= 1024, "barriers");

struct AfUnit {
    int r, bb, kvh, sp;
    int64_t tok[2];  // first token of each tile
    int64_t lo;      // first key block of this part
    int n[2];        // key blocks of each tile
    int64_t len;     // keys of the batch element
    int64_t pos0;    // position of query token 0; beyond every key when not causal
};

__device__ __forceinline__ AfUnit af_unit(const AttnFwdArgs& a, int64_t u)
{
    const AttnShape& s = a.s;
    AfUnit t;
    const int64_t v = div_fast(u, a.splits);
    t.sp = int(u - v * a.splits);
    const int64_t h = div_fast(v, a.q_blocks);
    int64_t qb = v - h * a.q_blocks;
    if (s.causal) qb = a.q_blocks - 1 - qb;  // the longest rows first
    int r = 0;
    while (r + 1 < s.W && h >= s.head_begin[r + 1]) ++r;
    t.r = r;
    const int local = int(h) - s.head_begin[r];
    t.bb = local / s.m[r];
    t.kvh = local - t.bb * s.m[r];
    t.len = s.Skv;
    if (s.kv_lens) t.len = min(s.Skv, int64_t(max(0, s.kv_lens[t.bb])));
    t.pos0 = s.causal ? (s.q_start ? int64_t(s.q_start[t.bb]) : 0) : s.Skv;
    int64_t blocks[2];
    for (int k = 0; k < 2; ++k) {
        t.tok[k] = (qb * 2 + k) * a.tile_tokens;
        const int64_t last = min(t.tok[k] + a.tile_tokens, s.Sq) - 1;
        int64_t keys = min(t.len, t.pos0 + last + 1);
        if (t.tok[k] >= s.Sq || keys < 0) keys = 0;
        blocks[k] = (keys + kAttnRows - 1) / kAttnRows;
    }
    const int64_t total = max(blocks[0], blocks[1]);
    const int64_t per = (total + a.splits - 1) / a.splits;
    t.lo = t.sp * per;
    const int64_t hi = min(total, t.lo + per);
    for (int k = 0; k < 2; ++k) t.n[k] = int(max(int64_t(0), min(blocks[k], hi) - t.lo));
    return t;
}

template <int DP, bool F16>
__global__ void __launch_bounds__(kAfThreads, 1)
    attn_fwd_kernel(const __grid_constant__ AttnFwdArgs a)
{
    using L = AfSmem<DP>;
    using E = ElemT<F16>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    AfBars& bars = *reinterpret_cast<AfBars*>(smem);
    volatile int* dead = &bars.dead;
    const AttnShape& s = a.s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (s.d + 15) / 16;      // steps of 16 along the head dimension
    const int halves = (s.d + 63) / 64;  // tiles of 64 columns

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars.q_full[t], 1);
            mbar_init(&bars.q_empty[t], 1);
            mbar_init(&bars.s_full[t], 1);
            mbar_init(&bars.p_ready[t], 4);
            mbar_init(&bars.o_full[t], 1);
            mbar_init(&bars.o_free[t], 4);
            mbar_init(&bars.o_staged[t], 4);
        }
        for (int k = 0; k < L::kStages; ++k) {
            mbar_init(&bars.kv_full[k], 1);
            mbar_init(&bars.kv_empty[k], 1);
        }
        mbar_init(&bars.drain, 1);
        bars.dead = 0;
        fence_barrier_init();
    }
    if (warp == kAfMmaWarp) tmem_alloc(&bars.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp == kAfLoadWarp) {
        if (lane == 0) {
            StageRing ring;
            uint32_t uses[2] = {0, 0};
            int64_t issued = 0;
            const uint32_t q_bytes = uint32_t(halves) * a.tile_tokens * s.group * 128u;
            const uint32_t kv_bytes = uint32_t(halves) * L::kHalf;
            bool ok = true;
            for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
                const AfUnit t = af_unit(a, u);
                for (int k = 0; ok && k < 2; ++k) {
                    if (t.n[k] == 0) continue;
                    if (uses[k] > 0) ok = wait_or_dead(&bars.q_empty[k], (uses[k] - 1) & 1, dead);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars.q_full[k], q_bytes);
                    for (int h = 0; h < halves; ++h)
                        tensor_g2s_4d(smem + L::kQ + k * L::kTile + h * L::kHalf, &a.qmap[t.r],
                                      64 * h, t.kvh * s.group, int(t.tok[k]), t.bb, &bars.q_full[k]);
                    ++uses[k];
                }
                const int n = max(t.n[0], t.n[1]);
                for (int j = 0; ok && j < 2 * n; ++j) {  // K0 V0 K1 V1 ...
                    if (issued >= L::kStages)
                        ok = wait_or_dead(&bars.kv_empty[ring.s], ring.phase ^ 1u, dead);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars.kv_full[ring.s], kv_bytes);
                    const CUtensorMap* map = (j & 1) ? &a.vmap[t.r] : &a.kmap[t.r];
                    for (int h = 0; h < halves; ++h)
                        tensor_g2s_4d(smem + L::kRing + ring.s * L::kTile + h * L::kHalf, map, 64 * h,
                                      t.kvh, int((t.lo + (j >> 1)) * kAttnRows), t.bb,
                                      &bars.kv_full[ring.s]);
                    ++issued;
                    ring.next(L::kStages);
                }
            }
            // leave no copy into this CTA's shared memory in flight
            for (int64_t k = max(int64_t(0), issued - L::kStages); k < issued; ++k)
                if (!mbar_wait_bounded(&bars.kv_full[k % L::kStages], uint32_t((k / L::kStages) & 1)))
                    atomicOr(&g_attn_fwd_status, kStatusDrainTimeout);
            for (int k = 0; k < 2; ++k)
                if (uses[k] > 0 && !mbar_wait_bounded(&bars.q_full[k], (uses[k] - 1) & 1))
                    atomicOr(&g_attn_fwd_status, kStatusDrainTimeout);
        }
        __syncwarp();
    } else if (warp == kAfMmaWarp) {
        const uint32_t id_s = tc_idesc(F16, kAttnRows, false);
        const uint32_t id_o = tc_idesc(F16, 16 * nk, true);
        const uint32_t q_at = smem_u32(smem + L::kQ), ring_at = smem_u32(smem + L::kRing);
        StageRing ring;
        uint32_t uses[2] = {0, 0}, blocks[2] = {0, 0};
        bool ok = true;
        auto all = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_or_dead(bar, parity, dead));
        };
        auto scores = [&](int t, uint32_t k_addr) {  // S_t = Q_t K^T
            for (int ks = 0; ks < nk; ++ks) {
                const uint32_t off = (ks >> 2) * L::kHalf + (ks & 3) * 32;
                tc_mma_ss(tmem + kAfS + t * 128, tc_desc_k(q_at + t * L::kTile + off),
                          tc_desc_k(k_addr + off), id_s, ks > 0);
            }
            tc_commit(&bars.s_full[t]);
        };
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            const AfUnit t = af_unit(a, u);
            const int n = max(t.n[0], t.n[1]);
            if (n == 0) continue;
            for (int k = 0; ok && k < 2; ++k)
                if (t.n[k] > 0) ok = all(&bars.q_full[k], uses[k] & 1);
            ok = ok && all(&bars.kv_full[ring.s], ring.phase);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                for (int k = 0; k < 2; ++k)
                    if (t.n[k] > 0) scores(k, ring_at + ring.s * L::kTile);
                tc_commit(&bars.kv_empty[ring.s]);
            }
            ring.next(L::kStages);
            for (int j = 0; ok && j < n; ++j) {
                const int vs = ring.s;
                ok = all(&bars.kv_full[vs], ring.phase);
                if (!ok) break;
                // A masked probability is zero, but zero times whatever lies past the last key
                // may be NaN: the block's rows past it become zeros.
                const int64_t past = t.len - (t.lo + j) * kAttnRows;
                if (past < kAttnRows && t.len < s.Skv) {
                    const int rows = kAttnRows - int(past), words = rows * 8;
                    for (int h = 0; h < halves; ++h)
                        for (int w = lane; w < words; w += 32)
                            st_shared_v4(smem + L::kRing + vs * L::kTile + h * L::kHalf +
                                             int(past) * 128 + w * 16,
                                         make_uint4(0, 0, 0, 0));
                    fence_proxy_async_shared();
                    __syncwarp();
                }
                ring.next(L::kStages);
                const int ks_stage = ring.s;
                const bool more = j + 1 < n;
                if (more) {
                    ok = all(&bars.kv_full[ks_stage], ring.phase);
                    if (!ok) break;
                    ring.next(L::kStages);
                }
                for (int k = 0; ok && k < 2; ++k) {
                    if (j >= t.n[k]) continue;
                    ok = all(&bars.p_ready[k], blocks[k] & 1);
                    ++blocks[k];
                    if (ok && j == 0 && uses[k] > 0) ok = all(&bars.o_free[k], (uses[k] - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t v_addr = ring_at + vs * L::kTile;
                        for (int ks = 0; ks < kAttnRows / 16; ++ks)
                            tc_mma_ts(tmem + kAfO + k * 128, tmem + kAfS + k * 128 + ks * 8,
                                      tc_desc_mn(v_addr + ks * 2048, L::kHalf), id_o,
                                      j > 0 || ks > 0);
                        if (j + 1 < t.n[k])
                            scores(k, ring_at + ks_stage * L::kTile);
                        else
                            tc_commit(&bars.o_full[k]);
                    }
                }
                if (ok && lane == 0) {
                    tc_commit(&bars.kv_empty[vs]);
                    if (more) tc_commit(&bars.kv_empty[ks_stage]);
                }
                __syncwarp();
            }
            for (int k = 0; k < 2; ++k) uses[k] += t.n[k] > 0;
        }
        // every product complete before tensor memory is given back
        if (lane == 0) {
            tc_commit(&bars.drain);
            if (!mbar_wait_bounded(&bars.drain, 0)) atomicOr(&g_attn_fwd_status, kStatusDrainTimeout);
        }
        __syncwarp();
    } else if (warp == kAfStoreWarp) {
        if (lane == 0) {
            uint32_t uses[2] = {0, 0};
            bool ok = true;
            for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
                const AfUnit t = af_unit(a, u);
                for (int k = 0; ok && k < 2; ++k) {
                    if (t.n[k] == 0) continue;
                    ok = wait_or_dead(&bars.o_staged[k], uses[k] & 1, dead);
                    if (!ok) break;
                    if (a.splits == 1) {
                        for (int h = 0; h < halves; ++h)
                            tensor_s2g_4d(&a.omap[t.r], 64 * h, t.kvh * s.group, int(t.tok[k]), t.bb,
                                          smem + L::kQ + k * L::kTile + h * L::kHalf);
                        bulk_commit();
                        bulk_wait_read<0>();
                    }
                    mbar_arrive(&bars.q_empty[k]);
                    ++uses[k];
                }
            }
            bulk_wait<0>();
        }
        __syncwarp();
    } else {  // softmax: tile w = warp / 4, one row a thread
        const int tile = warp >> 2;
        const int row = threadIdx.x & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t s_at = tmem + lanes + kAfS + tile * 128;
        const uint32_t o_at = tmem + lanes + kAfO + tile * 128;
        const int tok_in = row / s.group, head_in = row - tok_in * s.group;
        const float sl2 = s.scale * 1.4426950408889634f;  // scores to powers of two
        uint8_t* stage = smem + L::kQ + tile * L::kTile + row * 128;
        uint32_t uses = 0, blocks = 0;
        bool ok = true;
        auto all = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_or_dead(bar, parity, dead));
        };
        for (int64_t u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
            const AfUnit t = af_unit(a, u);
            const int64_t tok = t.tok[tile] + tok_in;
            const bool valid = tok_in < a.tile_tokens && tok < s.Sq;
            const int n = t.n[tile];
            // this row's log-sum-exp, and its row over all ranks
            const int64_t row_r =
                (int64_t(t.bb) * s.n[t.r] + t.kvh * s.group + head_in) * s.Sq + tok;
            const int64_t row_all = s.row_begin[t.r] + row_r;
            float* lse = a.splits == 1 ? a.lse[t.r] + row_r
                                       : a.part_lse + t.sp * s.row_begin[s.W] + row_all;
            uint8_t* o_row = a.splits == 1
                                 ? a.o[t.r] + ((int64_t(t.bb) * s.Sq + tok) * s.n[t.r] +
                                               t.kvh * s.group + head_in) * s.d * 2
                                 : nullptr;
            if (n == 0) {  // nothing visible to any row of the tile
                if (valid) {
                    *lse = -INFINITY;
                    if (o_row)
                        for (int c = 0; c < s.d * 2; c += 16)
                            st_v4(o_row + c, make_uint4(0, 0, 0, 0));
                }
                continue;
            }
            const int64_t lim = min(t.len, t.pos0 + tok + 1);  // keys this row sees
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j) {
                ok = all(&bars.s_full[tile], blocks & 1);
                if (!ok) break;
                ++blocks;
                tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(s_at + q * 32, x[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_wait_ld(x[q]);
                const int64_t left = lim - (t.lo + j) * kAttnRows;  // visible keys of this block
                if (__any_sync(0xffffffffu, left < kAttnRows)) {
                    const int seen = int(max(int64_t(0), min(left, int64_t(kAttnRows))));
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (q * 32 + c >= seen) x[q][c] = 0xFF800000u;  // -infinity
                }
                float mx[4] = {m, m, m, m};
#pragma unroll
                for (int c = 0; c < 32; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], __uint_as_float(x[q][c]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool grow = (top - m) * sl2 > kAfRescale;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2((m - top) * sl2) : 1.0f;
                    if (grow) m = top;
                    l *= f;
                    if (j > 0) {
#pragma unroll
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
                const float base = m == -INFINITY ? 0.0f : -m * sl2;
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
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_ready[tile]);
            }
            if (!ok) break;
            ok = all(&bars.o_full[tile], uses & 1);
            if (!ok) break;
            tc_fence_after();
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // NaN stays NaN
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                uint32_t y[32];
                tmem_ld32(o_at + c * 32, y);
                tmem_wait_ld(y);
                if (a.splits == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = E::pack(__uint_as_float(y[8 * i + 2 * k]) * inv,
                                           __uint_as_float(y[8 * i + 2 * k + 1]) * inv);
                        const int word = (c & 1) * 4 + i;  // 16-byte word of the tile row
                        st_shared_v4(stage + (c >> 1) * L::kHalf + ((word ^ (row & 7)) << 4),
                                     make_uint4(w[0], w[1], w[2], w[3]));
                    }
                } else if (valid) {
                    float* dst = a.part_o + (t.sp * s.row_begin[s.W] + row_all) * s.d + c * 32;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c * 32 + i * 4 < s.d)
                            *reinterpret_cast<float4*>(dst + i * 4) = make_float4(
                                __uint_as_float(y[4 * i]) * inv, __uint_as_float(y[4 * i + 1]) * inv,
                                __uint_as_float(y[4 * i + 2]) * inv,
                                __uint_as_float(y[4 * i + 3]) * inv);
                }
            }
            if (valid) *lse = l == 0.0f ? -INFINITY : m * s.scale + logf(l);
            tc_fence_before();
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars.o_free[tile]);
                mbar_arrive(&bars.o_staged[tile]);
            }
            ++uses;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && bars.dead) atomicOr(&g_attn_fwd_status, kStatusWaitTimeout);
    if (warp == kAfMmaWarp) tmem_free(tmem);
}

// Joins the parts of the keys: one warp a row; lane c holds columns 4c .. 4c + 3.
template <bool F16>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnFwdArgs a)
{
    using E = ElemT<F16>;
    const AttnShape& s = a.s;
    const int64_t rows = s.row_begin[s.W];
    const int lane = threadIdx.x & 31;
    for (int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5); row < rows;
         row += int64_t(gridDim.x) * 4) {
        float top = -INFINITY;
        for (int p = 0; p < a.splits; ++p) top = fmaxf(top, a.part_lse[p * rows + row]);
        float sum = 0.0f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < a.splits; ++p) {
            const float z = a.part_lse[p * rows + row];
            if (z == -INFINITY) continue;  // an empty part wrote no output
            const float w = expf(z - top);
            sum += w;
            if (lane * 4 < s.d) {
                const float4 o =
                    *reinterpret_cast<const float4*>(a.part_o + (p * rows + row) * s.d + lane * 4);
                acc.x = fmaf(w, o.x, acc.x);
                acc.y = fmaf(w, o.y, acc.y);
                acc.z = fmaf(w, o.z, acc.z);
                acc.w = fmaf(w, o.w, acc.w);
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

// Parts of the keys: as many as still fit one wave of the SMs, each with four blocks of keys at
// least (a part costs its start, an fp32 output and a share of the join).
int attn_fwd_splits(const AttnShape& s, int64_t units, int sm_count)
{
    if (units <= 0) return 1;
    const int64_t blocks = (s.Skv + kAttnRows - 1) / kAttnRows;
    int64_t n = sm_count / units;
    if (n > blocks / 4) n = blocks / 4;
    if (n > 64) n = 64;
    return n < 2 ? 1 : int(n);
}

template <int DP, bool F16>
static cudaError_t af_launch(const AttnFwdArgs& a, cudaStream_t stream, int device, int grid)
{
    static std::atomic<unsigned long long> raised{0};
    const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0;
    constexpr int smem = AfSmem<DP>::kTotal + 1024;
    if (bit && !(raised.load() & bit)) {
        cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<DP, F16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit);
    }
    attn_fwd_kernel<DP, F16><<<grid, kAfThreads, smem, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.splits == 1) return e;
    const int64_t blocks = (a.s.row_begin[a.s.W] + 3) / 4;
    attn_join_kernel<F16><<<unsigned(blocks < 1 << 16 ? blocks : 1 << 16), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

// One launch over all ranks (and the join); `grid` CTAs at most. The shape, outputs, splits and
// their buffers are set in `a`.
cudaError_t attn_fwd_launch(AttnFwdArgs& a, const void* const* q, const void* const* k,
                            const void* const* v, cudaStream_t stream, int device, int grid)
{
    const AttnShape& s = a.s;
    if (a.units == 0) return cudaSuccess;
    for (int r = 0; r < s.W; ++r) {
        if (s.n[r] == 0) continue;
        if (!encode_head_map(&a.qmap[r], q[r], s.f16, s.d, s.n[r], s.Sq, s.b, s.group, a.tile_tokens) ||
            !encode_head_map(&a.omap[r], a.o[r], s.f16, s.d, s.n[r], s.Sq, s.b, s.group,
                             a.tile_tokens) ||
            (s.Skv > 0 &&
             (!encode_head_map(&a.kmap[r], k[r], s.f16, s.d, s.m[r], s.Skv, s.b, 1, kAttnRows) ||
              !encode_head_map(&a.vmap[r], v[r], s.f16, s.d, s.m[r], s.Skv, s.b, 1, kAttnRows))))
            return cudaErrorInvalidValue;
    }
    if (int64_t(grid) > a.units) grid = int(a.units);
    if (s.d <= 64)
        return s.f16 ? af_launch<64, true>(a, stream, device, grid)
                     : af_launch<64, false>(a, stream, device, grid);
    return s.f16 ? af_launch<128, true>(a, stream, device, grid)
                 : af_launch<128, false>(a, stream, device, grid);
}

cudaError_t attn_fwd_status(unsigned* status, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_attn_fwd_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_fwd_status, &zero, sizeof(unsigned));
}

}  // namespace uly
