// The paged latent cache: writing new tokens' rows (append) and reading a
// sequence's rows back in order (gather).  A cached row is [c | r], 512
// latent and 64 shared key channels in bf16.
#include "latent_tc.cuh"

namespace kda {

// Error word of this file's kernels (bit 0: cu_seqlens or a length broke its
// precondition; bit 1: a page index outside the cache).
__device__ unsigned int g_kda_latent_error = 0;

namespace {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Block 0 raises bit 0 for offsets that decrease or leave [0, T] (the rest of
// the kernel stays inside its buffers whatever they are).
__device__ __forceinline__ void check_offsets(const int32_t *cu, int N, int T) {
    if (!cu || blockIdx.x != 0) return;
    bool bad = false;
    for (int b = threadIdx.x; b < N; b += blockDim.x) bad |= cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > T;
    if (bad) atomicOr(&g_kda_latent_error, kErrWait);
}

// ---------------------------------------------------------------- append
// A warp a token: the row's 72 16-byte pieces are read once (lane l holds
// latent pieces l and 32 + l, lanes 0..7 one of the shared part), the sum of
// squares is a warp reduction in fp32, each value is rounded to bf16 once.
// Bound by HBM: 1,152 B in and out a token (66,048 tokens: 30 us, 75 % of the
// measured copy; two or four tokens a warp, and a grid that stays with the
// weights in registers, measured 31 to 34 us).
constexpr int kAppendThreads = 256;

__device__ __forceinline__ float sumsq8(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = bf2_to_f2(w[e]);
        s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
    }
    return s;
}
__device__ __forceinline__ uint4 scale8(uint4 u, float n, const float *w) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(w) + 1);
    const float2 x0 = bf2_to_f2(u.x), x1 = bf2_to_f2(u.y), x2 = bf2_to_f2(u.z), x3 = bf2_to_f2(u.w);
    return make_uint4(f2_to_bf2(make_float2(x0.x * n * a.x, x0.y * n * a.y)),
                      f2_to_bf2(make_float2(x1.x * n * a.z, x1.y * n * a.w)),
                      f2_to_bf2(make_float2(x2.x * n * b.x, x2.y * n * b.y)),
                      f2_to_bf2(make_float2(x3.x * n * b.z, x3.y * n * b.w)));
}

__global__ void __launch_bounds__(kAppendThreads)
latent_append_kernel(const uint4 *__restrict__ x, uint4 *__restrict__ cache, PagedRows pages,
                     const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ cu,
                     const float *__restrict__ norm_w, float eps, int N, int T) {
    const int64_t t_of_warp = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    tc::let_next_begin();
    tc::wait_for_previous();
    check_offsets(cu, N, T);
    if (t_of_warp >= T) return;
    const int t = (int)t_of_warp;
    // the row does not wait for the walk to its place
    const uint4 *src = x + (size_t)t * kRowChunks;
    uint4 a = __ldcs(src + lane), b = __ldcs(src + 32 + lane), c = make_uint4(0, 0, 0, 0);
    if (lane < 8) c = __ldcs(src + 64 + lane);
    const int s = seq_of_token(cu, N, t);
    if (s < 0) return;                     // behind the last sequence
    const int start = cu ? cu[s] : s, count = cu ? cu[s + 1] - start : 1;
    const long long pos = (long long)seq_lens[s] - count + (t - start);
    if (pos < 0 || pos >= pages.max_len()) {
        if (lane == 0) atomicOr(&g_kda_latent_error, kErrWait);
        return;
    }
    const int64_t row = pages.row(s, (int)pos);
    if (row < 0) {
        if (lane == 0) atomicOr(&g_kda_latent_error, kErrSlot);
        return;
    }
    if (norm_w) {
        const float ss = warp_sum(sumsq8(a) + sumsq8(b));
        const float n = 1.f / sqrtf(ss * (1.f / kLatent) + eps);
        a = scale8(a, n, norm_w + 8 * lane);
        b = scale8(b, n, norm_w + 256 + 8 * lane);
    }
    uint4 *dst = cache + (size_t)row * kRowChunks;
    dst[lane] = a;
    dst[32 + lane] = b;
    if (lane < 8) dst[64 + lane] = c;
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
    check_offsets(cu, N, T);
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

cudaError_t launch_latent_append(const void *x, void *cache, const int32_t *table,
                                 const int32_t *seq_lens, const int32_t *cu, const float *norm_w,
                                 float eps, int N, int64_t T, int64_t P, int page, int max_pages,
                                 cudaStream_t stream) {
    const unsigned blocks = (unsigned)((T * 32 + kAppendThreads - 1) / kAppendThreads);
    return tc::launch_early(latent_append_kernel, blocks, kAppendThreads, 0, stream, static_cast<const uint4 *>(x),
                            static_cast<uint4 *>(cache), paged_rows(table, P, page, max_pages), seq_lens, cu, norm_w,
                            eps, N, (int)T);
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
