// cache_append.cu -- new tokens' keys and values written to their places in the pages of a cache.
//
// Token i < counts[bb] of batch element bb goes to position j = starts[bb] + i: row j % page of page
// table[bb][j / page]. A byte move, 4 m d e bytes a token read and written, bound by memory; with one
// token a sequence by the launch. A warp takes 32 tokens of a rank's keys or values: a lane works out one
// token's place (the divisions and the table, once a token), then the warp moves the tokens' rows of
// m_r * d in 16-byte words, neighbouring lanes neighbouring words, several loads before their stores.
// Measured: 4 x 16,380 tokens at most (ragged) of 8 heads of 128, W = 4, in 45-47 us, 4.9-5.1 TB/s read and
// written (0.72-0.76 of the copy peak; a place worked out by every word's thread: 74 us); 256 sequences' one token, W = 8,
// in 6.7 us.
#include <cuda_runtime.h>

#include "../../include/ulysses.h"
#include "paged.h"
#include "ptx.cuh"

namespace uly {

static __device__ unsigned g_cache_append_status;

constexpr int kApThreads = 128;
constexpr int kApEach = 8;  // words of a lane at a time

// grid: x over groups of tokens, y = 2 r + (0: keys, 1: values)
__global__ void __launch_bounds__(kApThreads) cache_append_kernel(const __grid_constant__ AppendArgs a)
{
    const int lane = threadIdx.x & 31, warps = kApThreads / 32;
    const int64_t all = a.b * a.tokens, step = int64_t(gridDim.x) * warps * 32;
    for (int what = blockIdx.y; what < 2 * a.W; what += gridDim.y) {
        const int r = what >> 1;
        const uint8_t* src = a.src[what & 1][r];
        uint8_t* dst = a.dst[what & 1][r];
        const uint32_t words = a.words[r];
        if (words == 0) continue;
        // Rows shorter than a warp: several at a time; longer ones: one, 32 words at a time.
        const uint32_t rows = words < 32 ? 32 / words : 1;
        const uint32_t sub = words < 32 ? lane / words : 0, first = lane - sub * words;
        for (int64_t t0 = (int64_t(blockIdx.x) * warps + (threadIdx.x >> 5)) * 32; t0 < all; t0 += step) {
            int64_t place = -1;  // row of the pool that the lane's token goes to
            const int64_t tok = t0 + lane, bb = tok < all ? div_fast(tok, a.tokens) : 0;
            const int64_t i = tok - bb * a.tokens;
            if (tok < all && !(a.counts && i >= a.counts[bb])) {
                const int64_t j = int64_t(a.starts[bb]) + i;
                const int64_t p = j < 0 ? -1 : div_fast(j, a.page);
                const int64_t page = p >= 0 && p < a.table_pages ? a.table[bb * a.table_pages + p] : -1;
                if (page >= 0 && page < a.pages)
                    place = page * a.page + (j - p * a.page);
                else
                    atomicOr(&g_cache_append_status, kStatusBadPage);
            }
            uint32_t t = sub, w = first;
            while (__any_sync(0xffffffffu, t < 32)) {
                uint4 x[kApEach];
                int64_t to[kApEach];
#pragma unroll
                for (int k = 0; k < kApEach; ++k) {
                    const int64_t row = __shfl_sync(0xffffffffu, place, t & 31);
                    to[k] = -1;
                    if (t < 32 && row >= 0 && sub < rows && w < words) {
                        to[k] = row * words + w;
                        x[k] = ld_stream_v4(src + ((t0 + t) * words + w) * 16);
                    }
                    w += 32;
                    if (words < 32 || w - first >= words) w = first, t += rows;
                }
#pragma unroll
                for (int k = 0; k < kApEach; ++k)
                    if (to[k] >= 0) st_v4(dst + to[k] * 16, x[k]);
            }
        }
    }
}

cudaError_t cache_append_launch(const AppendArgs& a, cudaStream_t stream, int64_t cap, int sm_count)
{
    constexpr int kTokens = kApThreads;  // of a CTA
    int64_t x = (a.b * a.tokens + kTokens - 1) / kTokens, y = 2 * a.W;
    const int64_t waves = int64_t(sm_count) * 16 * 4;  // four waves of full SMs
    if (x > waves) x = waves;
    if (x * y > cap) {
        if (y > cap) y = cap;
        x = cap / y;
    }
    cache_append_kernel<<<dim3(unsigned(x), unsigned(y)), kApThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t cache_append_status(unsigned* status, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_cache_append_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_cache_append_status, &zero, sizeof(unsigned));
}

}  // namespace uly
