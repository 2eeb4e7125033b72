// Absorbed latent attention of one or a few new tokens a sequence over the
// 4-bit paged cache, on the CUDA cores.
//
// A block a (token, head), its warps take every eighth position: lane l holds
// group l's 16 latent channels of the query and of the output and two of the
// shared part, a score is a warp reduction, maximum and sum run along; the
// warps' parts are joined in shared memory in order.
#include "latent4.cuh"
#include "latent_tc.cuh"

namespace kda {

// Error word of this file's kernels (bit 0: cu_seqlens or a length broke its
// precondition; bit 1: a page index outside the cache).
__device__ unsigned int g_kda_latent4_decode_error = 0;

namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps)
latent4_decode_kernel(const __nv_bfloat16 *__restrict__ q, const uint8_t *__restrict__ cache, PagedRows pages,
                      const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ cu, float scale_log2,
                      float unit, __nv_bfloat16 *__restrict__ o, float *__restrict__ lse, int N, int T, int H) {
    __shared__ float part[kWarps][kLatent];
    __shared__ float top[kWarps], sum[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x / H;
    tc::let_next_begin();
    tc::wait_for_previous();
    if (cu && blockIdx.x == 0) {
        bool bad = false;
        for (int b = threadIdx.x; b < N; b += blockDim.x) bad |= cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > T;
        if (bad) atomicOr(&g_kda_latent4_decode_error, kErrWait);
    }
    if (blockIdx.x == 0) {
        bool bad = false;
        for (int b = threadIdx.x; b < N; b += blockDim.x) bad |= seq_lens[b] < 0 || seq_lens[b] > pages.max_len();
        if (bad) atomicOr(&g_kda_latent4_decode_error, kErrWait);
    }
    const int s = seq_of_token(cu, N, t);
    if (s < 0) return;                     // no sequence's
    const int start = cu ? cu[s] : s, count = cu ? cu[s + 1] - start : 1;
    const int len = max(0, min(seq_lens[s], pages.max_len()));
    const int seen = min(len, len - count + (t - start) + 1);
    float x[16], acc[16], xr[2];
    const __nv_bfloat16 *row_q = q + (size_t)blockIdx.x * kLatentRow;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] = __bfloat162float(row_q[16 * lane + i]);
        acc[i] = 0.f;
    }
    xr[0] = __bfloat162float(row_q[kLatent + 2 * lane]);
    xr[1] = __bfloat162float(row_q[kLatent + 2 * lane + 1]);
    float m = -tc::kHuge, l = 0.f;
    for (int pos = warp; pos < seen; pos += kWarps) {
        const int64_t row = pages.row(s, pos);
        if (row < 0 && lane == 0) atomicOr(&g_kda_latent4_decode_error, kErrSlot);
        uint2 codes = make_uint2(0u, 0u);
        uint32_t sc = 0u, pe = 0u;
        if (row >= 0) {
            const uint8_t *p = cache + (size_t)row * kLatent4Row;
            codes = reinterpret_cast<const uint2 *>(p)[lane];
            sc = p[k4Scales + lane];
            pe = reinterpret_cast<const uint32_t *>(p + k4Pe)[lane];
        }
        const float g = __low2float(scales2(sc)) * unit;
        float c[16], dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = __half22float2(codes2(((i < 4 ? codes.x : codes.y) >> (8 * (i & 3))) & 0xffu));
            c[2 * i] = f.x * g;
            c[2 * i + 1] = f.y * g;
            dot = fmaf(x[2 * i], c[2 * i], fmaf(x[2 * i + 1], c[2 * i + 1], dot));
        }
        const float2 r = bf2_to_f2(pe);
        dot = fmaf(xr[0], r.x, fmaf(xr[1], r.y, dot));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        const float v = dot * scale_log2;
        const float now = fmaxf(m, v), f = exp2f(m - now), w = exp2f(v - now);
        m = now;
        l = l * f + w;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = fmaf(w, c[i], acc[i] * f);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) part[warp][16 * lane + i] = acc[i];
    if (lane == 0) {
        top[warp] = m;
        sum[warp] = l;
    }
    __syncthreads();
    float best = top[0], total = 0.f;
    for (int w = 1; w < kWarps; ++w) best = fmaxf(best, top[w]);
    for (int w = 0; w < kWarps; ++w) total += sum[w] * exp2f(top[w] - best);
    for (int ch = threadIdx.x; ch < kLatent; ch += 32 * kWarps) {
        float a = 0.f;
        for (int w = 0; w < kWarps; ++w) a += part[w][ch] * exp2f(top[w] - best);
        o[(size_t)blockIdx.x * kLatent + ch] = __float2bfloat16_rn(seen > 0 ? a / total : 0.f);
    }
    if (lse && threadIdx.x == 0)
        lse[blockIdx.x] = seen > 0 ? (best + log2f(total)) * 0.6931471805599453f : -CUDART_INF_F;
}

}  // namespace

size_t latent4_decode_workspace_bytes(int, int64_t, int) { return 0; }

cudaError_t launch_latent4_decode(const void *q, const void *cache, const int32_t *table,
                                  const int32_t *seq_lens, const int32_t *cu, float scale, int exponent,
                                  void *o, float *lse, int N, int64_t T, int H, int64_t P, int page,
                                  int max_pages, void *, cudaStream_t stream) {
    return tc::launch_early(latent4_decode_kernel, (unsigned)(T * H), 32 * kWarps, 0, stream,
                            static_cast<const __nv_bfloat16 *>(q), static_cast<const uint8_t *>(cache),
                            paged_rows(table, P, page, max_pages), seq_lens, cu, scale * 1.4426950408889634f,
                            pow2(exponent), static_cast<__nv_bfloat16 *>(o), lse, N, (int)T, H);
}

cudaError_t read_latent4_decode_error(unsigned int *code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kda_latent4_decode_error, sizeof(unsigned int));
    if (e != cudaSuccess || !reset) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kda_latent4_decode_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
