// Shared pieces of the latent-attention kernels: row sizes and the walk from
// packed tokens and positions to sequences and cache pages.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

constexpr int kLatent = kLatentDim;
constexpr int kLatentRow = kLatentDim + kLatentPeDim;
constexpr int kRowChunks = kLatentRow * 2 / 16;   // 16-byte pieces of a bf16 row: 72

// The paged cache as the kernels see it: rows of 576 bf16, `page` (a power of
// two, 1 << page_log2) of them a page, P pages; table[b][i] is the page that
// holds positions i * page .. of sequence b.
struct PagedRows {
    const int32_t *table;
    int64_t P;
    int page_log2;
    int max_pages;

    __device__ __forceinline__ int max_len() const {
        const long long m = (long long)max_pages << page_log2;
        return m > 0x7ffff000LL ? 0x7ffff000 : (int)m;   // sums with a tile stay in 32 bits
    }
    // Flat cache row of position `pos` of sequence `b`, or -1 (page index
    // outside the cache).  0 <= pos < max_len().
    __device__ __forceinline__ int64_t row(int b, int pos) const {
        const int32_t pg = table[(size_t)b * max_pages + (pos >> page_log2)];
        if (pg < 0 || pg >= P) return -1;
        return ((int64_t)pg << page_log2) + (pos & ((1 << page_log2) - 1));
    }
};

inline PagedRows paged_rows(const int32_t *table, int64_t P, int page, int max_pages) {
    int lg = 0;
    while ((1 << lg) < page) ++lg;
    return PagedRows{table, P, lg, max_pages};
}

// The sequence that holds packed token t: the largest b with cu[b] <= t.
// cu == nullptr: one token a sequence.  Returns -1 for a token that no
// sequence holds (behind the last one, or a broken cu).
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int N, int t) {
    if (!cu) return t < N ? t : -1;
    int lo = 0, hi = N;                   // cu[lo] <= t, cu[hi] > t unless t is past the end
    if (t < cu[0] || t >= cu[N]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return (cu[lo] <= t && t < cu[lo + 1]) ? lo : -1;
}

}  // namespace kda
