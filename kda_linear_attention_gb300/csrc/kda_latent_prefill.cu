// Causal attention of many new tokens with expanded keys and values: the
// prefill side of latent attention.
//
// Head h of token j has the key [kv[j][h][0:128] | k_pe[j]] and the value
// kv[j][h][128:256]; the last 64 key channels are one row a token for all
// heads.  The queries of a sequence are its last tokens: query i of nq sees
// keys 0 .. nk - nq + i.
//   s = scale <q, k>,   o = softmax(s) v,   lse = ln sum e^s
#include <math_constants.h>

#include "kda_internal.h"
#include "latent_common.cuh"

namespace kda {

// Error word of this file's kernels (bit 0: cu_seqlens broke its
// precondition).
__device__ unsigned int g_kda_latent_prefill_error = 0;

namespace {

constexpr int kThreads = 128;
constexpr int kTile = 64;

// A block a (token, head) row: scores of 64 keys, two threads a key, then a
// value column a thread.
__global__ void __launch_bounds__(kThreads)
latent_prefill_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ kv,
                      const __nv_bfloat16 *__restrict__ k_pe, int64_t pe_stride,
                      const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, float scale,
                      int causal, __nv_bfloat16 *__restrict__ o, float *__restrict__ lse, int N, int Tq,
                      int Tk, int H) {
    const int t = (int)(blockIdx.x / (unsigned)H), h = (int)(blockIdx.x % (unsigned)H);
    const int tid = threadIdx.x;
    const int s = seq_of_token(cu_q, N, t);
    if (s < 0) return;
    const int q0 = cu_q[s], nq = cu_q[s + 1] - q0;
    int k0 = cu_k[s], nk = cu_k[s + 1] - k0;
    if (k0 < 0 || nk < 0 || (int64_t)k0 + nk > Tk) {
        if (tid == 0) atomicOr(&g_kda_latent_prefill_error, kErrWait);
        nk = 0;
    }
    const int seen = causal ? max(0, nk - nq + (t - q0) + 1) : nk;
    __shared__ float sq[192], sc[kTile];
    const size_t row = blockIdx.x;
    for (int i = tid; i < 192; i += kThreads) sq[i] = __bfloat162float(q[row * 192 + i]);
    float m = -CUDART_INF_F, l = 0.f, acc = 0.f;
    for (int p0 = 0; p0 < seen; p0 += kTile) {
        const int n = min(kTile, seen - p0);
        __syncthreads();
        const int j = tid >> 1, half = tid & 1;
        float d = 0.f;
        if (j < n) {
            const size_t tok = (size_t)k0 + p0 + j;
            const __nv_bfloat16 *kr = kv + (tok * H + h) * 256;
            const __nv_bfloat16 *pr = k_pe + tok * pe_stride;
            for (int i = half; i < 128; i += 2) d = fmaf(sq[i], __bfloat162float(kr[i]), d);
            for (int i = half; i < 64; i += 2) d = fmaf(sq[128 + i], __bfloat162float(pr[i]), d);
        }
        d += __shfl_xor_sync(0xffffffffu, d, 1);
        if (half == 0) sc[j] = d * scale;
        __syncthreads();
        float mt = m;
        for (int i = 0; i < n; ++i) mt = fmaxf(mt, sc[i]);
        const float a = m == -CUDART_INF_F ? 0.f : expf(m - mt);
        l *= a;
        acc *= a;
        m = mt;
        for (int i = 0; i < n; ++i) {
            const float p = expf(sc[i] - m);
            l += p;
            acc = fmaf(p, __bfloat162float(kv[(((size_t)k0 + p0 + i) * H + h) * 256 + 128 + tid]), acc);
        }
    }
    o[row * 128 + tid] = __float2bfloat16_rn(l > 0.f ? acc / l : 0.f);
    if (lse && tid == 0) lse[row] = l > 0.f ? m + logf(l) : -CUDART_INF_F;
}

}  // namespace

cudaError_t launch_latent_prefill(const void *q, const void *kv, const void *k_pe, int64_t pe_stride,
                                  const int32_t *cu_q, const int32_t *cu_k, float scale, bool causal,
                                  void *o, float *lse, int N, int64_t Tq, int64_t Tk, int H,
                                  cudaStream_t stream) {
    latent_prefill_kernel<<<(unsigned)(Tq * H), kThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(kv),
        static_cast<const __nv_bfloat16 *>(k_pe), pe_stride, cu_q, cu_k, scale, causal ? 1 : 0,
        static_cast<__nv_bfloat16 *>(o), lse, N, (int)Tq, (int)Tk, H);
    return cudaGetLastError();
}

cudaError_t read_latent_prefill_error(unsigned int *code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kda_latent_prefill_error, sizeof(unsigned int));
    if (e != cudaSuccess || !reset) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kda_latent_prefill_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
