// cache_append.cu -- new tokens' keys and values written to their places in the pages of a cache.
//
// Token i < counts[bb] of batch element bb goes to position j = starts[bb] + i: row j % page of page
// table[bb][j / page]. A byte move, 4 m d e bytes a token read and written, bound by memory; with one
// token a sequence by the launch. A thread moves 16-byte words, four at a time with every load before
// the first store; neighbouring threads take neighbouring words, so a token's m_r * d row is read and
// written in whole lines.
#include <cuda_runtime.h>

#include "../../include/ulysses.h"
#include "paged.h"
#include "ptx.cuh"

namespace uly {

static __device__ unsigned g_cache_append_status;

constexpr int kApThreads = 256;
constexpr int kApEach = 4;  // words of a thread at a time

// grid: x over words, y = 2 r + (0: keys, 1: values)
__global__ void __launch_bounds__(kApThreads) cache_append_kernel(const __grid_constant__ AppendArgs a)
{
    for (int what = blockIdx.y; what < 2 * a.W; what += gridDim.y) {
        const int r = what >> 1, t = what & 1;
        const uint32_t words = a.words[r];
        const int64_t total = a.b * a.tokens * words;
        const uint8_t* src = a.src[t][r];
        uint8_t* dst = a.dst[t][r];
        for (int64_t at = int64_t(blockIdx.x) * (kApThreads * kApEach); at < total;
             at += int64_t(gridDim.x) * (kApThreads * kApEach)) {
            uint4 x[kApEach];
            int64_t to[kApEach];
#pragma unroll
            for (int k = 0; k < kApEach; ++k) {
                const int64_t w = at + k * kApThreads + threadIdx.x;
                to[k] = -1;
                if (w >= total) continue;
                const int64_t tok = div_fast(w, words), word = w - tok * words;
                const int64_t bb = div_fast(tok, a.tokens), i = tok - bb * a.tokens;
                if (a.counts && i >= a.counts[bb]) continue;
                const int64_t j = int64_t(a.starts[bb]) + i;
                const int64_t p = j < 0 ? -1 : div_fast(j, a.page);
                const int64_t page = p >= 0 && p < a.table_pages ? a.table[bb * a.table_pages + p] : -1;
                if (page < 0 || page >= a.pages) {
                    atomicOr(&g_cache_append_status, kStatusBadPage);
                    continue;
                }
                to[k] = (page * a.page + (j - p * a.page)) * words + word;
                x[k] = ld_stream_v4(src + w * 16);
            }
#pragma unroll
            for (int k = 0; k < kApEach; ++k)
                if (to[k] >= 0) st_v4(dst + to[k] * 16, x[k]);
        }
    }
}

cudaError_t cache_append_launch(const AppendArgs& a, cudaStream_t stream, int64_t cap, int sm_count)
{
    int64_t most = 0;
    for (int r = 0; r < a.W; ++r)
        if (a.words[r] > most) most = a.words[r];
    int64_t x = (a.b * a.tokens * most + kApThreads * kApEach - 1) / (kApThreads * kApEach);
    if (x == 0) return cudaSuccess;
    int64_t y = 2 * a.W;
    const int64_t waves = int64_t(sm_count) * 8 * 4;  // four waves of full SMs
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
