// The paged latent cache: writing new tokens' rows (append) and reading a
// sequence's rows back in order (gather).  A cached row is [c | r], 512
// latent and 64 shared key channels in bf16.
#include "latent_rows.cuh"

namespace kda {

// Error word of this file's kernels (bit 0: cu_seqlens or a length broke its
// precondition; bit 1: a page index outside the cache).
__device__ unsigned int g_kda_latent_error = 0;

namespace {

// ---------------------------------------------------------------- append
// A warp a token: the row's 72 16-byte pieces are read once (lane l holds
// latent pieces l and 32 + l, lanes 0..7 one of the shared part), the sum of
// squares is a warp reduction in fp32, each value is rounded to bf16 once.
// 1,152 B in and out a token (66,048 tokens: 30 us, 75 % of the measured copy;
// two or four tokens a warp, and a grid that stays with the weights in registers,
// measured 31 to 34 us).  With the shared part rotated, a pair a lane, 32 us: no
// limit is reached (325 instructions a token fill 66 % of the issue slots, DRAM is
// at 53 %, the first-level cache, which has the norm's weights for every token, at
// 64 %), and half of a warp's waiting is for its loads.
constexpr int kAppendThreads = 256;

template <bool ROTATED>
__global__ void __launch_bounds__(kAppendThreads)
latent_append_kernel(const uint4 *__restrict__ x, uint4 *__restrict__ cache, PagedRows pages,
                     const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ cu,
                     const float *__restrict__ norm_w, float eps, const Rotation rot, int N, int T) {
    const int64_t t_of_warp = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    tc::let_next_begin();
    tc::wait_for_previous();
    check_offsets(cu, N, T, &g_kda_latent_error);
    if (t_of_warp >= T) return;
    const int t = (int)t_of_warp;
    // the row does not wait for the walk to its place
    const uint4 *src = x + (size_t)t * kRowChunks;
    uint4 a = __ldcs(src + lane), b = __ldcs(src + 32 + lane), c = make_uint4(0, 0, 0, 0);
    uint32_t pe = 0u;
    if (ROTATED) pe = load_pair(reinterpret_cast<const __nv_bfloat16 *>(src + 64), lane, rot.interleaved);
    else if (lane < 8) c = __ldcs(src + 64 + lane);
    const NewRow at = new_row(pages, seq_lens, cu, N, t, lane, &g_kda_latent_error);
    if (at.row < 0) return;
    if (norm_w) {
        const float ss = warp_sum(sumsq8(a) + sumsq8(b));
        const float n = 1.f / sqrtf(ss * (1.f / kLatent) + eps);
        a = scale8(a, n, norm_w + 8 * lane);
        b = scale8(b, n, norm_w + 256 + 8 * lane);
    }
    uint4 *dst = cache + (size_t)at.row * kRowChunks;
    dst[lane] = a;
    dst[32 + lane] = b;
    if (ROTATED)
        store_pair(reinterpret_cast<__nv_bfloat16 *>(dst + 64), lane, rot.interleaved,
                   turned_pair(pe, rotation_of(rot, lane, at.pos)));
    else if (lane < 8) dst[64 + lane] = c;
}

// ---------------------------------------------------------------- gather
// A warp copies four consecutive rows: 288 16-byte pieces, nine a lane, all
// in flight at once; lanes 0..3 walk to the four source rows.  Bound by HBM:
// 1,152 B in and out a row (66,048 rows: 26 us, 87 % of the measured copy).
constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads)
latent_gather_kernel(const uint4 *__restrict__ cache, PagedRows pages, const int32_t *__restrict__ cu,
                     uint4 *__restrict__ out, int N, int T) {
    const int64_t t0 = 4 * ((int64_t)blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5));
    const int lane = threadIdx.x & 31;
    tc::let_next_begin();
    tc::wait_for_previous();
    check_offsets(cu, N, T, &g_kda_latent_error);
    if (t0 >= T) return;
    // source row of output row t0 + lane; -2: no such row, -1: its page is bad
    long long src = -2;
    if (lane < 4 && t0 + lane < T) {
        const int t = (int)t0 + lane;
        const int s = seq_of_token(cu, N, t);
        if (s >= 0) {
            const int pos = t - cu[s];
            if (pos < pages.max_len()) src = pages.row(s, pos);
            else src = -1;
            if (src < 0) atomicOr(&g_kda_latent_error, pos < pages.max_len() ? kErrSlot : kErrWait);
        }
    }
    uint4 v[9];
    long long from[9];
#pragma unroll
    for (int i = 0; i < 9; ++i) {
        const int e = 32 * i + lane;
        from[i] = __shfl_sync(0xffffffffu, src, e / kRowChunks);
        v[i] = make_uint4(0, 0, 0, 0);
        if (from[i] >= 0) v[i] = __ldcs(cache + (size_t)from[i] * kRowChunks + e % kRowChunks);
    }
    uint4 *dst = out + (size_t)t0 * kRowChunks;
#pragma unroll
    for (int i = 0; i < 9; ++i)
        if (from[i] > -2) dst[32 * i + lane] = v[i];
}

}  // namespace

namespace {

template <bool ROTATED>
cudaError_t launch_append(const void *x, void *cache, const int32_t *table, const int32_t *seq_lens,
                          const int32_t *cu, const float *norm_w, float eps, const Rotation &rot, int N, int64_t T,
                          int64_t P, int page, int max_pages, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((T * 32 + kAppendThreads - 1) / kAppendThreads);
    return tc::launch_early(latent_append_kernel<ROTATED>, blocks, kAppendThreads, 0, stream,
                            static_cast<const uint4 *>(x), static_cast<uint4 *>(cache),
                            paged_rows(table, P, page, max_pages), seq_lens, cu, norm_w, eps, rot, N, (int)T);
}

}  // namespace

cudaError_t launch_latent_append(const void *x, void *cache, const int32_t *table,
                                 const int32_t *seq_lens, const int32_t *cu, const float *norm_w,
                                 float eps, int N, int64_t T, int64_t P, int page, int max_pages,
                                 cudaStream_t stream) {
    return launch_append<false>(x, cache, table, seq_lens, cu, norm_w, eps, Rotation{nullptr, 1.f, false}, N, T, P,
                                page, max_pages, stream);
}

cudaError_t launch_latent_append_rotated(const void *x, void *cache, const int32_t *table,
                                         const int32_t *seq_lens, const int32_t *cu, const float *norm_w,
                                         float eps, const Rotation &rot, int N, int64_t T, int64_t P,
                                         int page, int max_pages, cudaStream_t stream) {
    return launch_append<true>(x, cache, table, seq_lens, cu, norm_w, eps, rot, N, T, P, page, max_pages, stream);
}

cudaError_t launch_latent_gather(const void *cache, const int32_t *table, const int32_t *cu, void *out,
                                 int N, int64_t T, int64_t P, int page, int max_pages,
                                 cudaStream_t stream) {
    const unsigned blocks = (unsigned)(((T + 3) / 4 * 32 + kGatherThreads - 1) / kGatherThreads);
    return tc::launch_early(latent_gather_kernel, blocks, kGatherThreads, 0, stream,
                            static_cast<const uint4 *>(cache), paged_rows(table, P, page, max_pages), cu,
                            static_cast<uint4 *>(out), N, (int)T);
}

cudaError_t read_latent_error(unsigned int *code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kda_latent_error, sizeof(unsigned int));
    if (e != cudaSuccess || !reset) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kda_latent_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
