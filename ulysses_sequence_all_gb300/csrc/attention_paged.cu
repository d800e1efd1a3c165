// attention_paged.cu -- attention of the last few tokens of each sequence over a key-value cache held
// in pages (or, without a table, over contiguous keys and values), with or without a sliding window.
//
// The query at position p sees the keys j < len with j <= p and (j > p - window or j < sinks). Per row
// o = sum_j exp(s_j - m) v_j / l and lse = m + log l as in attention_fwd.cuh; a row that sees no key
// gives zeros and -infinity.
//
// With R = group * tokens query rows a key head, each 4 d bytes of a key and its value carry 4 d R
// flops: below some 200 rows memory bounds it, and the design is made to keep copies in flight. All the
// work (the blocks of 64 keys that any row of a (batch element, key head) sees) is laid end
// to end and cut into as many equal shares as CTAs run at a time, two an SM, whatever the sequences'
// lengths: a CTA finds its share from the lengths by one scan. Warp 4 walks the share and copies block
// after block into a ring (tensor maps, a lane a page, the table read a block ahead); warps 0-3 take 16
// keys of a block each and wait for no one but the copies until a sequence ends. There the warps'
// maxima, sums and outputs are joined through the last block's stage; a sequence that several CTAs share
// leaves its parts as normalised fp32 outputs with their lse, which attn_paged_join_kernel adds in order:
// the same bits from run to run.
//
// Measured (bf16, copy peak 6,767 GB/s): one token each on 16 caches of 12,000-32,768 tokens, 32 heads over 4 of
// 128 in 115-117 us (0.92 of the peak), on 256 of 100-2,000, 64 heads over 8, in 170-171 us (0.89), with a window of
// 4,096 on 32 sequences, 40 heads over 8, in 92-94 us (0.86); four drafted tokens on 8 caches of 3,000-9,000 in
// 39-41 us (0.65), one short cache in 9.3 us: about 10 us of each are the launches, the first copies' chain of
// loads (lengths, table, map, keys) and the last join. 32 rows on the 16 caches take 120 us.
//
// Products: S^T = K Q^T and O^T += V^T P^T with keys (and columns of V) as the 16 rows of an
// m16n8k16 product, so that a tile of 8 query rows costs no more than its own work. A product of this
// size reads its fragments straight from the tiles that the copies left and keeps its sums in
// registers; the fifth generation's 128 rows and the trip through tensor memory take longer up to 16 or 32 rows
// (kPagedFewRows). P^T's fragments are S^T's
// transposed, 8x8 blocks at a time.
// P is rounded to the element type (fp16: times 2^7, so that many keys of little weight are not lost),
// relative to a maximum that may lag by 2^8; maxima, sums and outputs are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "../../include/ulysses.h"
#include "attention.h"
#include "fused_row.cuh"
#include "paged.h"
#include "tensor_map.h"

namespace uly {

static __device__ unsigned g_attn_paged_status;

constexpr int kPgThreads = 2 * 32 * kPagedWarps;  // warps 0-3, and a warpgroup with the copying one
// Registers a thread: 256 x 128 at launch = 128 x this + 128 x (256 - this), what the roles take
template <int DP, int RT>
constexpr int kPgRegsProducts = DP == 128 ? (RT == 2 ? 200 : 184) : 176;
constexpr float kPgRescale = 8.0f;  // log2 of the growth of a row's maximum that forces a rescale
constexpr float kPgUpF16 = 7.0f;    // fp16 probabilities are held times 2^this
constexpr int kPgJoinThreads = 256, kPgJoinParts = 8;
// What a sequence's end (its join, the next one's queries) costs a CTA, in blocks of keys, by the kernel's query
// rows. 1, 2, 3 with 8 rows: one token on 256 sequences of 100-2,000 keys 166, 170, 171 us, of 100-200 keys 47,
// 46, 46, on 8 of 3,000-9,000 38, 37, 37 (0: the first two 191 and 58 when the end was slower). 2, 3, 4, 7 with 16
// rows on the first 186, 187, 192, 199, four tokens on the last 41, 39, 39, 39; 3, 4, 5, 7 with 32 rows on the first
// 228, 217, 218, 225.
constexpr int pg_end(int rows) { return rows <= 8 ? 2 : rows <= 16 ? 3 : 4; }

// ---- what there is to do ----------------------------------------------------------------------------

// A batch element: the keys that its rows see, and the blocks that hold them.
struct PagedEntry {
    int bb;
    int n;              // blocks, one at least: rows that see no key are written as well
    int first, near;    // the first tokens' blocks 0 .. first - 1; the others from block `near` on
    int snk, lo, end;   // some row sees key j: j < snk, or lo <= j < end
    int len;
    int64_t pos0;       // position of query token 0
    __device__ __forceinline__ int block(int j) const { return j < first ? j : near + j - first; }
    __device__ __forceinline__ bool sees(int a, int b) const  // any of keys a .. b - 1
    {
        return a < end && (min(b, end) > lo || a < snk);
    }
};

__device__ __forceinline__ PagedEntry paged_entry(const PagedArgs& a, int bb)
{
    PagedEntry t;
    t.bb = bb;
    t.len = a.kv_lens ? max(0, min(a.kv_lens[t.bb], a.room)) : a.room;
    t.pos0 = a.q_start ? int64_t(a.q_start[t.bb]) : a.from_end ? t.len - a.Sq : 0;
    t.end = int(max(int64_t(0), min(int64_t(t.len), t.pos0 + a.Sq)));
    t.lo = int(max(int64_t(0), min(int64_t(t.end), t.pos0 + 1 - a.window)));
    t.snk = min(a.sinks, t.lo);
    t.near = t.lo / kPagedBlock;
    t.first = min((t.snk + kPagedBlock - 1) / kPagedBlock, t.near);
    t.n = max(1, t.first + (t.end + kPagedBlock - 1) / kPagedBlock - t.near);
    return t;
}

// The way through a share's blocks: entry by entry, in an entry head by head (the heads of a token lie
// next to one another), in a head block by block.
struct PagedWalk {
    int64_t left;  // of the share, from the sequence's beginning (its end included) on
    int e, head, j;
    PagedEntry en;
    __device__ __forceinline__ bool more(const PagedArgs& a) const { return left > j + a.end; }
    // blocks of the sequence that are the share's: j .. stop() - 1
    __device__ __forceinline__ int stop(const PagedArgs& a) const { return int(min(int64_t(en.n), left - a.end)); }
    __device__ __forceinline__ void step(const PagedArgs& a)
    {
        if (++j < en.n) return;
        j = 0;
        left -= en.n + a.end;
        if (++head < a.m_begin[a.W]) return;
        head = 0;
        if (more(a)) en = paged_entry(a, ++e);
    }
};

// The work is measured in blocks, a sequence (of one head) of n as `end` + n, its end first:
// equal shares of that are equal times, however short the sequences are. A share that begins inside an end
// begins with the sequence.
__device__ __forceinline__ int64_t paged_share(int64_t total, int parts, int64_t c)  // where it begins
{
    const int64_t q = total / parts, rem = total - q * parts;
    return c * q + min(c, rem);
}

__device__ __forceinline__ int paged_owner(int64_t total, int parts, int64_t at)
{
    const int64_t q = total / parts, rem = total - q * parts, big = rem * (q + 1);
    return int(at < big ? at / (q + 1) : rem + (at - big) / q);
}

// ---- the kernel -------------------------------------------------------------------------------------

template <int DP>
struct PgSmem {
    static constexpr int kHalf = kPagedBlock * 128;           // 64 columns of a block
    static constexpr int kV = kHalf * (DP / 64);              // values after keys
    static constexpr int kBlock = 2 * kV;
    static constexpr int kStages = DP == 128 ? 3 : 6;
    static constexpr int kRing = 2048;                        // PgShared first
    static constexpr int kTotal = kRing + kStages * kBlock;
    static_assert(2 * (kTotal + 1024 + kSmemReservedPerCta) <= kSmemPerSm, "two CTAs an SM");
};

struct PgShared {
    uint64_t full[6], empty[6];
    float2 ml[kPagedWarps][16];  // each warp's maxima and sums
    int used[kPagedWarps];       // whether it has outputs
    int64_t warp_sum[kPgThreads / 32];
    int64_t before;  // blocks of the entries before `entry`
    int entry;
};
static_assert(sizeof(PgShared) <= 2048, "shared memory");

template <bool F16>
__device__ __forceinline__ void pg_mma(float (&c)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}

// Four 8x8 blocks of 16-bit elements; lane l gives the address of row l % 8 of block l / 8.
template <bool TRANS>
__device__ __forceinline__ void pg_ldmatrix(uint32_t (&x)[4], uint32_t addr)
{
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(addr)
                     : "memory");
}

__device__ __forceinline__ uint32_t pg_transpose(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A limit of nothing (the self-test's) is one look: a copy takes less time than the hardware may hold a try_wait
// back for, so that no wait would ever run out.
__device__ __forceinline__ bool pg_wait(uint64_t* bar, uint32_t parity, uint64_t limit)
{
    if (mbar_test_wait(bar, parity)) return true;
    if (limit == 0) return false;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > limit) return false;
    return true;
}

__device__ __forceinline__ void pg_sync()  // the four warps with products
{
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kPagedWarps) : "memory");
}

// RT: tiles of 8 query rows of a warp. RH: groups of such rows; warps w with the same w % RH share a group
// and part the block's four tiles of keys between them.
template <int DP, bool F16, int RT, int RH>
__global__ void __launch_bounds__(kPgThreads, 2)
    attn_paged_kernel(const __grid_constant__ PagedArgs a)
{
    using L = PgSmem<DP>;
    using E = ElemT<F16>;
    constexpr int K = L::kStages, kD = DP / 16;
    constexpr int kMine = 8 * RT, kRows = kMine * RH;  // query rows of a warp, of the kernel
    constexpr int kPartRows = 2048 / (DP * 4);         // rows of outputs in 16 rows of a tile's 128 bytes
    constexpr float kUp = F16 ? kPgUpF16 : 0.0f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    PgShared& sh = *reinterpret_cast<PgShared*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int halves = (a.d + 63) / 64, heads = a.m_begin[a.W];
    const uint64_t limit = uint64_t(a.wait_us) * 1000u;

    if (threadIdx.x == 0) {
        for (int k = 0; k < K; ++k) {
            mbar_init(&sh.full[k], 1);
            mbar_init(&sh.empty[k], kPagedWarps);
        }
        fence_barrier_init();
    }

    // How many blocks there are, and in which entry a share begins.
    const int each = (a.b - 1) / kPgThreads + 1;
    const int e0 = min(a.b, int(threadIdx.x) * each), e1 = e0 + min(each, a.b - e0);
    int64_t mine = 0;
    for (int e = e0; e < e1; ++e) mine += paged_entry(a, e).n + a.end;
    int64_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kPgThreads / 32; ++w) {
        if (w < warp) upto += sh.warp_sum[w];
        total += sh.warp_sum[w];
    }
    total *= heads;

    StageRing ring;
    int64_t issued = 0;  // warp 4: blocks copied
    bool ok = true;

    // Share c: its blocks begin .. stop - 1, and the walk through them. Called by every warp.
    int64_t begin = 0, stop = 0;
    PagedWalk walk;
    auto share = [&](int c) {
        begin = paged_share(total, a.parts, c);
        stop = paged_share(total, a.parts, c + 1);
        __syncthreads();
        if (begin >= (upto - mine) * heads && begin < upto * heads) {
            int64_t at = upto - mine;
            int e = e0;
            for (int n; begin >= (at + (n = paged_entry(a, e).n + a.end)) * heads; ++e) at += n;
            sh.entry = e;
            sh.before = at;
        }
        __syncthreads();
        walk.left = walk.j = 0;
        if (begin < stop) {
            walk.e = sh.entry;
            walk.en = paged_entry(a, walk.e);
            const int64_t off = begin - sh.before * heads;
            walk.head = int(div_fast(off, walk.en.n + a.end));
            const int x = int(off - int64_t(walk.head) * (walk.en.n + a.end));
            walk.j = max(0, x - a.end);
            walk.left = stop - begin + x;
        }
    };

    if (warp >= kPagedWarps) {  // the copies
        regs_shrink<256 - kPgRegsProducts<DP, RT>>();
        if (warp > kPagedWarps && lane < a.W && a.n[lane] > 0)  // (the first copies else wait for them)
            prefetch_map(warp & 1 ? &a.kmap[lane] : &a.vmap[lane]);
        for (int c = blockIdx.x; c < a.parts; c += gridDim.x) {
            share(c);
            if (warp > kPagedWarps) continue;
            const int box = lane * a.box;  // this lane's rows of a block
            bool seen = false;             // some row sees one of them; their page, its row
            int page = 0, row = 0, r = 0, kvh = 0;
            bool live = false;             // a block is in hand
            auto look = [&]() {            // the walk's next block that any row sees anything of
                live = false;
                while (walk.more(a)) {
                    const int key0 = walk.en.block(walk.j) * kPagedBlock;
                    live = walk.en.sees(key0, key0 + kPagedBlock);
                    if (live) {
                        r = 0;
                        while (r + 1 < a.W && walk.head >= a.m_begin[r + 1]) ++r;
                        kvh = walk.head - a.m_begin[r];
                        const int key = key0 + box;
                        seen = box < kPagedBlock && walk.en.sees(key, key + a.box);
                        page = walk.en.bb;
                        row = key;
                        if (a.table && seen) {
                            const int p = int(uint32_t(key) / uint32_t(a.page));
                            page = a.table[int64_t(walk.en.bb) * a.table_pages + p];
                            row = key - p * a.page;
                        }
                    }
                    walk.step(a);
                    if (live) break;
                }
            };
            look();
            while (live && ok) {
                const bool now_seen = seen;
                const int now_page = page, now_row = row, now_r = r, now_kvh = kvh;
                look();
                if (issued >= K)
                    ok = __all_sync(0xffffffffu,
                                    pg_wait(&sh.empty[ring.s], ring.phase ^ 1u, limit));
                if (!ok) break;
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, now_seen));
                uint64_t* bar = &sh.full[ring.s];
                if (lane == 0) mbar_arrive_expect_tx(bar, boxes * uint32_t(a.box) * 256u * halves);
                __syncwarp();
                if (now_seen) {
                    // (outside the pool a copy reads zeros)
                    if (now_page < 0 || now_page >= a.pages)
                        atomicOr(&g_attn_paged_status, kStatusBadPage);
                    uint8_t* to = smem + L::kRing + ring.s * L::kBlock + box * 128;
                    for (int h = 0; h < halves; ++h) {
                        tensor_g2s_4d(to + h * L::kHalf, &a.kmap[now_r], 64 * h, now_kvh, now_row,
                                      now_page, bar);
                        tensor_g2s_4d(to + L::kV + h * L::kHalf, &a.vmap[now_r], 64 * h, now_kvh, now_row,
                                      now_page, bar);
                    }
                }
                __syncwarp();
                ++issued;
                ring.next(K);
            }
        }
        if (!ok && lane == 0) atomicOr(&g_attn_paged_status, kStatusWaitTimeout);
        // leave no copy into this CTA's shared memory in flight
        if (lane == 0)
            for (int64_t k = max(int64_t(0), issued - K); k < issued; ++k)
                if (!mbar_wait_bounded(&sh.full[k % K], uint32_t((k / K) & 1)))
                    atomicOr(&g_attn_paged_status, kStatusDrainTimeout);
        let_next_start();
        return;
    }

    // the products
    regs_grow<kPgRegsProducts<DP, RT>>();
    const float sl2 = a.scale * 1.4426950408889634f;
    const int quad = lane >> 2, pair = (lane & 3) * 2;  // fragments: key (column of V); query row
    for (int c = blockIdx.x; c < a.parts; c += gridDim.x) {
        share(c);
        PagedShared shared = {0, 0, 0, 0};
        uint32_t q[RT][kD][2];
        // The walk's rank and key head; this warp's queries of it.
        auto place = [&](int* r, int* kvh) {
            *r = 0;
            while (*r + 1 < a.W && walk.head >= a.m_begin[*r + 1]) ++*r;
            *kvh = walk.head - a.m_begin[*r];
        };
        auto queries = [&]() {
            int r, kvh;
            place(&r, &kvh);
            const int row0 = (warp % RH) * kMine, row_end = int(a.Sq) * a.group;
            auto query = [&](int row) {  // its first byte
                const int tok = int(uint32_t(row) / uint32_t(a.group));
                return a.q[r] + ((int64_t(walk.en.bb) * a.Sq + tok) * a.n[r] + kvh * a.group + row -
                                 tok * a.group) * a.d * 2;
            };
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int row = row0 + t * 8 + quad;
                const uint8_t* src = query(row) + pair * 2;
#pragma unroll
                for (int ks = 0; ks < kD; ++ks)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        q[t][ks][h] = 0;
                        if (row < row_end && ks * 16 + h * 8 < a.d)
                            q[t][ks][h] =
                                __ldg(reinterpret_cast<const uint32_t*>(src + (ks * 16 + h * 8) * 2));
                    }
            }
        };
        if (walk.more(a)) queries();
        while (walk.more(a)) {
            const PagedEntry en = walk.en;
            int r, kvh;
            place(&r, &kvh);
            const int head = walk.head, from = walk.j, to_block = walk.stop(a);
            const int64_t place = int64_t(walk.e) * heads + head;
            const int64_t at_end = stop - walk.left + a.end + en.n;  // where the sequence ends in the work
            // (fewer than 2^27 rows; no 64-bit divisions: see the join)
            const int row0 = (warp % RH) * kMine, row_end = int(a.Sq) * a.group;
            // keys that every row sees: below hi_all, and from lo_all on or first tokens
            const int hi_all = int(max(int64_t(0), min(int64_t(en.len), en.pos0 + 1)));
            const int lo_all = int(max(int64_t(0), min(int64_t(en.len), en.pos0 + a.Sq - a.window)));
            float m[RT][2], l[RT][2], o[RT][kD][4];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
#pragma unroll
                for (int i = 0; i < 2; ++i) m[t][i] = -INFINITY, l[t][i] = 0.0f;
#pragma unroll
                for (int i = 0; i < kD; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[t][i][x] = 0.0f;
            }
            bool used = false;  // this warp has seen keys of the sequence
            int stage = -1;     // of the sequence's last block here, held until its outputs are joined
            for (int j = from; j < to_block; ++j) {
                const int block0 = en.block(j) * kPagedBlock;
                if (ok && en.sees(block0, block0 + kPagedBlock)) {
                    ok = __all_sync(0xffffffffu, pg_wait(&sh.full[ring.s], ring.phase, limit));
                    if (!ok) continue;
                    stage = ring.s;
                    ring.next(K);
#pragma unroll 1
                    for (int i = warp / RH; i < kPagedWarps; i += kPagedWarps / RH) {
                        const int key0 = block0 + i * kPagedTile;
                        uint8_t* keys = smem + L::kRing + stage * L::kBlock + i * (kPagedTile * 128);
                        if (!en.sees(key0, key0 + kPagedTile)) continue;
                        used = true;
                        const bool edge = key0 + kPagedTile > hi_all ||
                                          (key0 < lo_all && key0 + kPagedTile > a.sinks);
                        if (edge) {
                            // A masked probability is zero, but zero times what no row sees (or
                            // was not even copied) may be NaN.
                            for (int i = lane; i < kPagedTile * 8 * halves; i += 32) {
                                const int k = (i >> 3) & (kPagedTile - 1), h = i / (kPagedTile * 8);
                                if (!en.sees(key0 + k, key0 + k + 1))
                                    st_shared_v4(keys + L::kV + h * L::kHalf + k * 128 + (i & 7) * 16,
                                                 make_uint4(0, 0, 0, 0));
                            }
                            fence_proxy_async_shared();  // (before the next copy into this stage)
                            __syncwarp();
                        }
                        // S^T, in two sums (a sum of eight products waits for each of them). Columns past d are
                        // zeros in the copies and in q: all DP are taken, with no branch between the products.
                        float s[RT][4], s2[RT][4];
#pragma unroll
                        for (int t = 0; t < RT; ++t)
#pragma unroll
                            for (int x = 0; x < 4; ++x) s[t][x] = s2[t][x] = 0.0f;
                        const uint32_t keys_at = smem_u32(keys);
                        {
                            const int k = ((lane >> 3) & 1) * 8 + (lane & 7), w = lane >> 4;
#pragma unroll
                            for (int ks = 0; ks < kD; ++ks) {
                                uint32_t x[4];
                                pg_ldmatrix<false>(x, keys_at + (ks >> 2) * L::kHalf + k * 128 +
                                                          ((((ks & 3) * 2 + w) ^ (k & 7)) << 4));
#pragma unroll
                                for (int t = 0; t < RT; ++t)
                                    pg_mma<F16>((ks & 1) ? s2[t] : s[t], x, q[t][ks][0], q[t][ks][1]);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < RT; ++t)
#pragma unroll
                            for (int x = 0; x < 4; ++x) s[t][x] += s2[t][x];
                        if (edge) {
#pragma unroll
                            for (int t = 0; t < RT; ++t)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int row = row0 + t * 8 + pair + i;
                                    const int64_t p = en.pos0 + int(uint32_t(row) / uint32_t(a.group));
                                    const int hi = int(max(int64_t(0), min(int64_t(en.len), p + 1)));
                                    const int lo =
                                        int(max(int64_t(0), min(int64_t(en.len), p + 1 - a.window)));
#pragma unroll
                                    for (int x = 0; x < 2; ++x) {
                                        const int key = key0 + quad + 8 * x;
                                        if (key >= hi || (key < lo && key >= a.sinks))
                                            s[t][2 * x + i] = -INFINITY;
                                    }
                                }
                        }
                        bool grow = false;
#pragma unroll
                        for (int t = 0; t < RT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                grow |= (fmaxf(s[t][i], s[t][2 + i]) - m[t][i]) * sl2 > kPgRescale;
                        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                            for (int t = 0; t < RT; ++t) {
                                float f[2];
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float top = fmaxf(s[t][i], s[t][2 + i]);
#pragma unroll
                                    for (int x = 4; x < 32; x <<= 1)
                                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                                    const bool up = (top - m[t][i]) * sl2 > kPgRescale;
                                    f[i] = up ? ex2((m[t][i] - top) * sl2) : 1.0f;
                                    if (up) m[t][i] = top;
                                    l[t][i] *= f[i];
                                }
#pragma unroll
                                for (int i = 0; i < kD; ++i) {
                                    o[t][i][0] *= f[0], o[t][i][2] *= f[0];
                                    o[t][i][1] *= f[1], o[t][i][3] *= f[1];
                                }
                            }
                        }
                        uint32_t p[RT][2];
#pragma unroll
                        for (int t = 0; t < RT; ++t) {
                            float e[4];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float base = (m[t][i] == -INFINITY ? 0.0f : -m[t][i] * sl2) + kUp;
                                e[i] = ex2(fmaf(s[t][i], sl2, base));
                                e[2 + i] = ex2(fmaf(s[t][2 + i], sl2, base));
                                l[t][i] += e[i] + e[2 + i];
                            }
                            p[t][0] = pg_transpose(E::pack(e[0], e[1]));
                            p[t][1] = pg_transpose(E::pack(e[2], e[3]));
                        }
                        // O^T
                        {
                            const int k = (lane >> 4) * 8 + (lane & 7), w = (lane >> 3) & 1;
                            const uint32_t v_at = keys_at + L::kV + k * 128;
#pragma unroll
                            for (int i = 0; i < kD; ++i) {
                                uint32_t x[4];
                                pg_ldmatrix<true>(x, v_at + (i >> 2) * L::kHalf +
                                                         ((((i & 3) * 2 + w) ^ (k & 7)) << 4));
#pragma unroll
                                for (int t = 0; t < RT; ++t) pg_mma<F16>(o[t][i], x, p[t][0], p[t][1]);
                            }
                        }
                    }
                    const int next =
                        j + 1 < to_block ? en.block(j + 1) * kPagedBlock : en.end;
                    if (en.sees(next, next + kPagedBlock)) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.empty[stage]);
                        stage = -1;
                    }
                }
            }
            walk.j = to_block - 1;
            walk.step(a);
            if (walk.more(a)) queries();  // (they arrive during the join)

            // Join the warps: a row's maximum, sum and output.
            const bool whole = from == 0 && to_block == en.n;
            const int64_t part = 2 * int64_t(c) + (from == 0 ? 1 : 0);
            if (from == 0) {
                shared = {0, 0, 0, 0};
                if (!whole) shared = {paged_owner(total, a.parts, at_end - 1) - c + 1, c, en.bb, head};
                if (a.by_sequence && threadIdx.x == 0) a.shared[place] = shared;
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], x);
                    if (lane < 4) sh.ml[warp][t * 8 + pair + i] = make_float2(m[t][i], l[t][i]);
                }
            used = used && stage >= 0;  // (it has given up otherwise)
            if (lane == 0) sh.used[warp] = used;
            // Row `row` of warp w's outputs lies where tile w's keys and values of the last block were.
            if constexpr (RH > 1) pg_sync();  // (which other warps read as well)
            auto out_at = [&](int w, int row, int col) {
                return reinterpret_cast<float*>(smem + L::kRing + stage * L::kBlock +
                                                (row / kPartRows) * L::kHalf + w * (kPagedTile * 128)) +
                       (row % kPartRows) * DP + (col ^ (((row >> 1) & 3) << 3));
            };
            __syncwarp();
            if (used) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int i = 0; i < kD; ++i)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            *out_at(warp, t * 8 + pair + (x & 1), i * 16 + (x >> 1) * 8 + quad) = o[t][i][x];
            }
            pg_sync();
            // (rolled, and with 32-bit divisions: what the products' loop and a sequence's end do not both fit of
            // the instruction cache is fetched again at every end)
#pragma unroll 1
            for (int it = threadIdx.x; it < kRows * (DP / 8); it += 32 * kPagedWarps) {
                const int row = it / (DP / 8), col = it % (DP / 8) * 8;
                const int rh = row / kMine, in = row - rh * kMine;  // the warps' group, the row in it
                if (col >= a.d) continue;
                float top = -INFINITY, sum = 0.0f, y[8];
#pragma unroll
                for (int w = 0; w < kPagedWarps; w += RH) top = fmaxf(top, sh.ml[w + rh][in].x);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = 0.0f;
#pragma unroll
                for (int w = 0; w < kPagedWarps; w += RH) {
                    const float2 z = sh.ml[w + rh][in];
                    // (not by the maximum: scores that were all NaN leave that at minus infinity)
                    if (!sh.used[w + rh] || stage < 0 || z.y == 0.0f) continue;
                    const float f = ex2((z.x - top) * sl2);
                    sum = fmaf(f, z.y, sum);
#pragma unroll
                    for (int k = 0; k < 8; k += 4) {
                        const float4 v = *reinterpret_cast<const float4*>(out_at(w + rh, in, col + k));
                        y[k] = fmaf(f, v.x, y[k]);
                        y[k + 1] = fmaf(f, v.y, y[k + 1]);
                        y[k + 2] = fmaf(f, v.z, y[k + 2]);
                        y[k + 3] = fmaf(f, v.w, y[k + 3]);
                    }
                }
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // NaN stays NaN
                const float lse = sum == 0.0f ? -INFINITY
                                              : top * a.scale + (logf(sum) - kUp * 0.69314718056f);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] *= inv;
                if (!whole) {
                    const int64_t at_row = part * kRows + row;
                    float4* dst = reinterpret_cast<float4*>(a.part_o + at_row * a.d + col);
                    dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                    dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                    if (col == 0) a.part_lse[at_row] = lse;
                } else if (row < row_end) {
                    const int tok = int(uint32_t(row) / uint32_t(a.group));
                    const int h = kvh * a.group + (row - tok * a.group);
                    st_v4(a.o[r] + (((int64_t(en.bb) * a.Sq + tok) * a.n[r] + h) * a.d + col) * 2,
                          make_uint4(E::pack(y[0], y[1]), E::pack(y[2], y[3]), E::pack(y[4], y[5]),
                                     E::pack(y[6], y[7])));
                    if (col == 0) a.lse[r][(int64_t(en.bb) * a.n[r] + h) * a.Sq + tok] = lse;
                }
            }
            fence_proxy_async_shared();  // (a copy comes into this stage next)
            pg_sync();
            if (stage >= 0 && lane == 0) mbar_arrive(&sh.empty[stage]);
        }
        if (!a.by_sequence && threadIdx.x == 0) a.shared[c] = shared;
    }
    if (!ok && lane == 0) atomicOr(&g_attn_paged_status, kStatusWaitTimeout);
    let_next_start();
}

// Joins what several CTAs made of a sequence: block x looks at note x. `y_rows` of its warps take
// a row each, the others of a row every (warps / y_rows)-th part; a lane has 4 columns.
template <bool F16>
__global__ void __launch_bounds__(kPgJoinThreads, 2)
    attn_paged_join_kernel(const __grid_constant__ PagedArgs a, int y_rows)
{
    using E = ElemT<F16>;
    constexpr int kWarps = kPgJoinThreads / 32;
    __shared__ float4 acc_at[kWarps][32];
    __shared__ float2 ml_at[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ways = kWarps / y_rows, way = warp % ways;
    wait_for_previous();
    for (int note = blockIdx.x; note < a.notes; note += gridDim.x) {
        const PagedShared s = a.shared[note];
        if (s.parts == 0) continue;
        for (int row0 = blockIdx.y * y_rows; row0 < a.rows; row0 += gridDim.y * y_rows) {
            const int row = row0 + warp / ways;
            float top = -INFINITY, sum = 0.0f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            auto slot = [&](int p) {
                return (p == 0 ? 2 * int64_t(s.cta) + 1 : 2 * int64_t(s.cta + p)) * a.rows + row;
            };
            // eight parts at a time, all on their way at once, relative to the largest lse so far
            for (int p0 = way; p0 < s.parts; p0 += kPgJoinParts * ways) {
                float4 o[kPgJoinParts];
                float f[kPgJoinParts];
#pragma unroll
                for (int k = 0; k < kPgJoinParts; ++k) {
                    const int p = p0 + k * ways;
                    f[k] = -INFINITY;
                    o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (p >= s.parts) continue;
                    f[k] = a.part_lse[slot(p)];
                    if (lane * 4 < a.d)
                        o[k] = *reinterpret_cast<const float4*>(a.part_o + slot(p) * a.d + lane * 4);
                }
                float most = top;
#pragma unroll
                for (int k = 0; k < kPgJoinParts; ++k) most = fmaxf(most, f[k]);
                const float keep = top == -INFINITY ? 0.0f : expf(top - most);
                top = most;
                sum *= keep;
                acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
                for (int k = 0; k < kPgJoinParts; ++k) {
                    const float w = f[k] == -INFINITY ? 0.0f : expf(f[k] - top);  // (NaN stays NaN)
                    sum += w;
                    acc.x = fmaf(w, o[k].x, acc.x);
                    acc.y = fmaf(w, o[k].y, acc.y);
                    acc.z = fmaf(w, o[k].z, acc.z);
                    acc.w = fmaf(w, o[k].w, acc.w);
                }
            }
            if (ways > 1) {  // the ways of a row, in order
                acc_at[warp][lane] = acc;
                if (lane == 0) ml_at[warp] = make_float2(top, sum);
                __syncthreads();
                if (way == 0) {
                    float most = top;
                    for (int w = 1; w < ways; ++w) most = fmaxf(most, ml_at[warp + w].x);
                    acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    sum = 0.0f;
                    for (int w = 0; w < ways; ++w) {
                        const float2 z = ml_at[warp + w];
                        if (z.x == -INFINITY && z.y == 0.0f) continue;
                        const float f = expf(z.x - most);
                        const float4 y = acc_at[warp + w][lane];
                        sum = fmaf(f, z.y, sum);
                        acc.x = fmaf(f, y.x, acc.x);
                        acc.y = fmaf(f, y.y, acc.y);
                        acc.z = fmaf(f, y.z, acc.z);
                        acc.w = fmaf(f, y.w, acc.w);
                    }
                    top = most;
                }
                __syncthreads();
            }
            if (way != 0 || row >= int(a.Sq) * a.group) continue;
            int r = 0;
            while (r + 1 < a.W && s.head >= a.m_begin[r + 1]) ++r;
            const int tok = row / a.group;
            const int64_t h = int64_t(s.head - a.m_begin[r]) * a.group + (row - tok * a.group);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (lane * 4 < a.d)
                st_v2(a.o[r] + (((int64_t(s.bb) * a.Sq + tok) * a.n[r] + h) * a.d + lane * 4) * 2,
                      E::pack(acc.x * inv, acc.y * inv), E::pack(acc.z * inv, acc.w * inv));
            if (lane == 0)
                a.lse[r][(int64_t(s.bb) * a.n[r] + h) * a.Sq + tok] = sum == 0.0f ? top : top + logf(sum);
        }
    }
}

// ---- host -------------------------------------------------------------------------------------------

void attn_paged_split(PagedArgs* a, int sm_count)
{
    a->rows = 8;
    while (a->rows < a->Sq * a->group) a->rows *= 2;  // (kPagedFewRows at most)
    a->parts = 2 * sm_count;
    a->end = pg_end(a->rows);
    const int64_t all = int64_t(a->b) * a->m_begin[a->W];
    a->by_sequence = all <= a->parts;
    a->notes = int32_t(a->by_sequence ? all : a->parts);
}

template <int DP, bool F16, int RT, int RH>
static cudaError_t pg_launch(const PagedArgs& a, cudaStream_t stream, int device, int64_t cap)
{
    static std::atomic<unsigned long long> raised{0};
    const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0;
    constexpr int smem = PgSmem<DP>::kTotal + 1024;
    if (bit && !(raised.load() & bit)) {
        cudaError_t e = cudaFuncSetAttribute(attn_paged_kernel<DP, F16, RT, RH>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit);
    }
    const unsigned grid = unsigned(a.parts < cap ? a.parts : cap);
    attn_paged_kernel<DP, F16, RT, RH><<<grid, kPgThreads, smem, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // Few sequences are shared by many CTAs each: then a block has fewer rows, its warps more of the parts
    // (as many as they have on their way at once).
    int y_rows = kPgJoinThreads / 32;
    while (y_rows > 1 && int64_t(a.notes) * kPgJoinParts * (kPgJoinThreads / 32 / y_rows) < a.parts) y_rows /= 2;
    unsigned x = unsigned(a.notes < cap ? a.notes : cap), y = unsigned(a.rows / y_rows);
    if (int64_t(x) * y > cap) y = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(x, y);
    cfg.blockDim = dim3(kPgJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cap == kAttnMostCtas ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<F16>, a, y_rows);
}

template <int DP, bool F16>
static cudaError_t pg_launch_rows(const PagedArgs& a, cudaStream_t stream, int device, int64_t cap)
{
    if (a.rows == 8) return pg_launch<DP, F16, 1, 1>(a, stream, device, cap);
    if (a.rows == 16) return pg_launch<DP, F16, 2, 1>(a, stream, device, cap);
    return pg_launch<DP, F16, 2, 2>(a, stream, device, cap);
}

cudaError_t attn_paged_launch(PagedArgs& a, const void* const* k, const void* const* v,
                              cudaStream_t stream, int device, int64_t cap)
{
    if (a.m_begin[a.W] == 0) return cudaSuccess;
    for (int r = 0; r < a.W; ++r) {
        const int m = a.m_begin[r + 1] - a.m_begin[r];
        if (m == 0) continue;
        if (!encode_head_map(&a.kmap[r], k[r], a.f16, a.d, m, a.page, a.pages, 1, a.box) ||
            !encode_head_map(&a.vmap[r], v[r], a.f16, a.d, m, a.page, a.pages, 1, a.box))
            return cudaErrorInvalidValue;
    }
    if (a.d <= 64)
        return a.f16 ? pg_launch_rows<64, true>(a, stream, device, cap)
                     : pg_launch_rows<64, false>(a, stream, device, cap);
    return a.f16 ? pg_launch_rows<128, true>(a, stream, device, cap)
                 : pg_launch_rows<128, false>(a, stream, device, cap);
}

cudaError_t attn_paged_status(unsigned* status, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_attn_paged_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_paged_status, &zero, sizeof(unsigned));
}

}  // namespace uly
