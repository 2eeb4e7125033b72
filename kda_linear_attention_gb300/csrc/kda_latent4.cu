// The paged latent cache in 4 bits: writing new tokens' rows (append) and
// reading rows back as bf16 (gather).
#include "latent4.cuh"
#include "latent_rows.cuh"

namespace kda {

// Error word of this file's kernels (bit 0: cu_seqlens or a length broke its
// precondition; bit 1: a page index outside the cache).
__device__ unsigned int g_kda_latent4_error = 0;

namespace {

// ---------------------------------------------------------------- append
// A warp a token, a group of 16 channels a lane: the norm's sum is a warp
// reduction in the order of the bf16 append's (in another order a code or scale
// moved in 9 of 524,288 rows), a group's maximum and codes are the lane's own.
// The channels are rounded to bf16 first, so that a row stands for what the bf16
// cache would hold; scale and codes then follow from it without a further
// rounding: max / 6 and c / scale are quotients of numbers of 8 and 4 significant
// bits, which meet a border of e4m3 or e2m1 exactly or stay 2^-15 away from it,
// and both are exact where they meet one.
// 1,152 B in and 416 B out a token; bound by its instructions: 358 a token with
// rotation, 478 with the norm too, which fill 77 % of the issue slots while the SMs
// are active (DRAM 37 % and 28 %).  66,048 rows: 25 us, 28 with rotation (54 % of the
// measured copy), 35 with the norm, 37 with both (41 %); with divisions in the Newton
// step's place 36 where it is 28.
constexpr int kAppendThreads = 256;

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__global__ void __launch_bounds__(kAppendThreads)
latent4_append_kernel(const uint4 *__restrict__ x, uint8_t *__restrict__ cache, PagedRows pages,
                      const int32_t *__restrict__ seq_lens, const int32_t *__restrict__ cu,
                      const float *__restrict__ norm_w, float eps, const Rotation rot, float unit, int N, int T) {
    const int64_t t_of_warp = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    tc::let_next_begin();
    tc::wait_for_previous();
    check_offsets(cu, N, T, &g_kda_latent4_error);
    if (t_of_warp >= T) return;
    const int t = (int)t_of_warp;
    // the row does not wait for the walk to its place
    const uint4 *src = x + (size_t)t * kRowChunks;
    uint4 a = __ldcs(src + 2 * lane), b = __ldcs(src + 2 * lane + 1);
    uint32_t pe = load_pair(reinterpret_cast<const __nv_bfloat16 *>(src + 64), lane, rot.interleaved);
    const NewRow at = new_row(pages, seq_lens, cu, N, t, lane, &g_kda_latent4_error);
    if (at.row < 0) return;
    if (norm_w) {
        const float ss = warp_sum_of_neighbours(sumsq8(a), sumsq8(b), lane);
        const float n = 1.f / sqrtf(ss * (1.f / kLatent) + eps);
        a = scale8(a, n, norm_w + 16 * lane);
        b = scale8(b, n, norm_w + 16 * lane + 8);
    }
    float c[16];
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = bf2_to_f2(w[i]);
            c[2 * i] = f.x;
            c[2 * i + 1] = f.y;
        }
    }
    float top = fabsf(c[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = max_nan(top, fabsf(c[i]));
    // unit = 2^-exponent: its products are exact
    const __nv_fp8_storage_t s8 = __nv_cvt_float_to_fp8(top * unit / 6.f, __NV_SATFINITE, __NV_E4M3);
    const float s = __low2float(scales2(s8)) / unit;
    // a scale of 0 has codes of 0 (signed); of NaN, any
    const float r = s > 0.f ? 1.f / s : 0.f;
    const float most = 8.f * s;
    if (top > most && s > 0.f) {                    // past the last code (6), where c / s may be past fp32
#pragma unroll
        for (int i = 0; i < 16; ++i) c[i] = fmaxf(fminf(c[i], most), -most);
    }
    uint32_t code[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // c / s: one step of Newton's method on the product with the rounded reciprocal, which is off by
        // an ulp or two, makes a quotient exact that fp32 holds, as it does each border.  (The signs are
        // such that -0 stays -0.)
        float2 q = make_float2(c[2 * i] * r, c[2 * i + 1] * r);
        q.x = fmaf(-fmaf(q.x, s, -c[2 * i]), r, q.x);
        q.y = fmaf(-fmaf(q.y, s, -c[2 * i + 1]), r, q.y);
        const uint32_t two = __nv_cvt_float2_to_fp4x2(q, __NV_E2M1, cudaRoundNearest);
        code[i >> 2] |= two << (8 * (i & 3));
    }
    uint8_t *dst = cache + (size_t)at.row * kLatent4Row;
    reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(code[0], code[1]);
    dst[k4Scales + lane] = s8;
    if (rot.turns) pe = turned_pair(pe, rotation_of(rot, lane, at.pos));
    store_pair(reinterpret_cast<__nv_bfloat16 *>(dst + k4Pe), lane, rot.interleaved, pe);
}

// ---------------------------------------------------------------- gather
// A warp takes four consecutive rows, all their loads in flight at once; a lane
// turns four bytes of codes into 16 bytes of bf16, twice a row, so that both
// sides are whole lines.  Bound by HBM: 416 B in and 1,152 B out a row (66,048
// rows: 17 us, 90 % of the measured copy).
constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 4;

// eight codes of one scale as bf16 (exact: a code times a scale has 6 significant bits)
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t scale, float unit) {
    const __half2 s = __half2half2(__low2half(scales2(scale)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(__hmul2(codes2((codes >> (8 * i)) & 0xffu), s));
        w[i] = f2_to_bf2(make_float2(f.x * unit, f.y * unit));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kGatherThreads)
latent4_gather_kernel(const uint8_t *__restrict__ cache, PagedRows pages, const int32_t *__restrict__ cu,
                      uint4 *__restrict__ out, float unit, int N, int T) {
    const int64_t t0 = kGatherRows * ((int64_t)blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5));
    const int lane = threadIdx.x & 31;
    tc::let_next_begin();
    tc::wait_for_previous();
    check_offsets(cu, N, T, &g_kda_latent4_error);
    if (t0 >= T) return;
    // source row of output row t0 + lane; -2: no such row, -1: its page is bad
    long long src = -2;
    if (lane < kGatherRows && t0 + lane < T) {
        const int t = (int)t0 + lane;
        const int s = seq_of_token(cu, N, t);
        if (s >= 0) {
            const int pos = t - cu[s];
            if (pos < pages.max_len()) src = pages.row(s, pos);
            else src = -1;
            if (src < 0) atomicOr(&g_kda_latent4_error, pos < pages.max_len() ? kErrSlot : kErrWait);
        }
    }
    uint32_t code[kGatherRows][2], scale[kGatherRows][2];
    long long from[kGatherRows];
    uint4 pe = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
        from[i] = __shfl_sync(0xffffffffu, src, i);
        const uint8_t *row = cache + (size_t)(from[i] >= 0 ? from[i] : 0) * kLatent4Row;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            code[i][j] = scale[i][j] = 0u;
            if (from[i] >= 0) {
                code[i][j] = __ldcs(reinterpret_cast<const uint32_t *>(row) + 32 * j + lane);
                scale[i][j] = __ldcs(row + k4Scales + 16 * j + (lane >> 1));
            }
        }
        if (from[i] >= 0 && (lane >> 3) == i)   // eight lanes a row
            pe = __ldcs(reinterpret_cast<const uint4 *>(row + k4Pe) + (lane & 7));
    }
    uint4 *dst = out + (size_t)t0 * kRowChunks;
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
        if (from[i] == -2) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            dst[i * kRowChunks + 32 * j + lane] = values8(code[i][j], scale[i][j], unit);
        if ((lane >> 3) == i) dst[i * kRowChunks + 64 + (lane & 7)] = pe;
    }
}
static_assert(kGatherRows == 4, "eight lanes a row's shared part");

}  // namespace

cudaError_t launch_latent4_append(const void *x, void *cache, const int32_t *table, const int32_t *seq_lens,
                                  const int32_t *cu, const float *norm_w, float eps, const Rotation &rot,
                                  int exponent, int N, int64_t T, int64_t P, int page, int max_pages,
                                  cudaStream_t stream) {
    const unsigned blocks = (unsigned)((T * 32 + kAppendThreads - 1) / kAppendThreads);
    return tc::launch_early(latent4_append_kernel, blocks, kAppendThreads, 0, stream, static_cast<const uint4 *>(x),
                            static_cast<uint8_t *>(cache), paged_rows(table, P, page, max_pages), seq_lens, cu, norm_w,
                            eps, rot, pow2(-exponent), N, (int)T);
}

cudaError_t launch_latent4_gather(const void *cache, const int32_t *table, const int32_t *cu, void *out,
                                  int exponent, int N, int64_t T, int64_t P, int page, int max_pages,
                                  cudaStream_t stream) {
    const unsigned blocks = (unsigned)(((T + kGatherRows - 1) / kGatherRows * 32 + kGatherThreads - 1) / kGatherThreads);
    return tc::launch_early(latent4_gather_kernel, blocks, kGatherThreads, 0, stream,
                            static_cast<const uint8_t *>(cache), paged_rows(table, P, page, max_pages), cu,
                            static_cast<uint4 *>(out), pow2(exponent), N, (int)T);
}

cudaError_t read_latent4_error(unsigned int *code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kda_latent4_error, sizeof(unsigned int));
    if (e != cudaSuccess || !reset) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kda_latent4_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
