// C-ABI shim of libkda_gb300: argument validation and kernel dispatch.
// Declarations and the contract of each call are in include/kda.h.
#include <stdint.h>

#include <initializer_list>

#include "../../include/kda.h"
#include "kda_internal.h"

namespace {

constexpr int kVersion = 400;   // 0.4.0: rotary positions, the latent cache in 4 bits

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// 4-bit rows are read in sectors of 32 bytes.
bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// T tokens (>= 0) of H heads (>= 1): rows that 32 bits number.
bool rows_in_32_bits(int64_t T, int H) { return T < (int64_t(1) << 31) && T * H < (int64_t(1) << 31); }

// Sizes shared by the calls on a paged latent cache.
int latent_cache_dims(int N, int64_t T, int64_t P, int page, int max_pages, int d_latent, int d_pe) {
    if (d_latent != kda::kLatentDim || d_pe != kda::kLatentPeDim) return KDA_ERR_DIM;
    if (N < 1 || T < 0 || T >= (int64_t(1) << 31) || P < 1 || max_pages < 1) return KDA_ERR_DIM;
    if (page < 16 || page > 1024 || (page & (page - 1)) != 0) return KDA_ERR_DIM;
    if (P >= (int64_t(1) << 31) || P * page >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    return KDA_OK;
}

// The numbers of a rotation.
int rotation_status(float amplitude, int layout) {
    if (amplitude - amplitude != 0.f || (layout != KDA_ROTARY_HALF && layout != KDA_ROTARY_INTERLEAVED))
        return KDA_ERR_VALUE;
    return KDA_OK;
}

int exponent_status(int exponent) {
    return exponent < -kda::kLatent4Exponent || exponent > kda::kLatent4Exponent ? KDA_ERR_VALUE : KDA_OK;
}

// Strides of T x H rows of d elements of e bytes: whole 16 bytes, and all the
// rows within 2^60 elements, so that a row's place in bytes fits 63 bits.
bool row_strides(int64_t token, int64_t head, int64_t T, int H, int d, int64_t e) {
    const int64_t most = int64_t(1) << 31;    // T and H are below it too: no product passes 62 bits
    if (token < 0 || head < 0 || token >= most || head >= most || token * e % 16 != 0 || head * e % 16 != 0) return false;
    return T == 0 || (T - 1) * token + (H - 1) * head + d <= (int64_t(1) << 60);
}

}  // namespace

extern "C" {

int kda_version(void) { return kVersion; }

const char *kda_status_string(int status) {
    switch (status) {
        case KDA_OK: return "ok";
        case KDA_ERR_NULL: return "a required pointer is NULL";
        case KDA_ERR_DIM: return "unsupported or inconsistent sizes (dk = dv = 128, N >= 1, H >= 1; latent rows 512 + 64, page a power of two)";
        case KDA_ERR_CHUNK: return "chunk must be 16, 32 or 64";
        case KDA_ERR_ALIGN: return "a pointer is not aligned (16 bytes; 32 for a 4-bit cache; 256 for a workspace)";
        case KDA_ERR_DTYPE: return "dtype must be KDA_BF16 or KDA_F32";
        case KDA_ERR_WORKSPACE: return "workspace could not be allocated or is too small";
        case KDA_ERR_CUDA: return "CUDA launch error";
        case KDA_ERR_VALUE: return "a scalar argument is out of range (eps >= 0, finite q_scale, scale > 0)";
        default: return "unknown status";
    }
}

int kda_prefill_chunked(const void *q, const void *k, const void *v, const float *g,
                        const float *beta, const float *S0, float *o, float *S_out,
                        const int32_t *cu_seqlens, int N, int64_t T, int H, int dk, int dv,
                        int chunk, int dtype, void *stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (dk != kda::kDK || dv != kda::kDV || N < 1 || H < 1 || T < 0 || T >= (int64_t(1) << 31))
        return KDA_ERR_DIM;
    if ((int64_t)N * H * (kda::kDV / 32) >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (chunk != 16 && chunk != 32 && chunk != 64) return KDA_ERR_CHUNK;
    if (!S_out || !cu_seqlens) return KDA_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !g || !beta || !o)) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, g, beta, S0, o, S_out, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16 && chunk == 64 && T > 0) {
        const cudaError_t e = kda::launch_prefill_split(q, k, v, g, beta, S0, o, S_out, cu_seqlens,
                                                        N, T, H, s);
        return e == cudaErrorMemoryAllocation ? KDA_ERR_WORKSPACE : cuda_status(e);
    }
    return cuda_status(kda::launch_prefill_simt(q, k, v, g, beta, S0, o, S_out, cu_seqlens, N, T, H,
                                                chunk, dtype == KDA_BF16, s));
}

int kda_prefill_chunked_events(const void *q, const void *k, const void *v, const float *g,
                               const float *beta, const float *S0, float *o, float *S_out,
                               const int32_t *cu_seqlens, int N, int64_t T, int H, int dk, int dv,
                               int chunk, int dtype, void *stream, void *const *events) {
    if (!events || !events[0] || !events[1] || !events[2] || !events[3]) return KDA_ERR_NULL;
    if (dtype != KDA_BF16 || chunk != 64 || T <= 0) return KDA_ERR_CHUNK;
    if (dk != kda::kDK || dv != kda::kDV || N < 1 || H < 1 || T >= (int64_t(1) << 31))
        return KDA_ERR_DIM;
    if ((int64_t)N * H * (kda::kDV / 32) >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (!S_out || !cu_seqlens || !q || !k || !v || !g || !beta || !o) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, g, beta, S0, o, S_out, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    cudaEvent_t ev[4];
    for (int i = 0; i < 4; ++i) ev[i] = static_cast<cudaEvent_t>(events[i]);
    const cudaError_t e = kda::launch_prefill_split(q, k, v, g, beta, S0, o, S_out, cu_seqlens, N,
                                                    T, H, static_cast<cudaStream_t>(stream), ev);
    return e == cudaErrorMemoryAllocation ? KDA_ERR_WORKSPACE : cuda_status(e);
}

int kda_prefill_chunked_noalloc(const void *q, const void *k, const void *v, const float *g,
                                const float *beta, const float *S0, float *o, float *S_out,
                                const int32_t *cu_seqlens, int N, int64_t T, int H, int dk,
                                int dv, int chunk, int dtype, void *stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (dk != kda::kDK || dv != kda::kDV || N < 1 || H < 1 || T < 0 || T >= (int64_t(1) << 31))
        return KDA_ERR_DIM;
    if ((int64_t)N * H * (kda::kDV / 32) >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (chunk != 16 && chunk != 32 && chunk != 64) return KDA_ERR_CHUNK;
    if (!S_out || !cu_seqlens) return KDA_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !g || !beta || !o)) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, g, beta, S0, o, S_out, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16 && chunk == 64 && T > 0) {
        if (kda::prefill_split_workspace_bytes(N, T, H) > kda::kNoAllocScratchBytes)
            return KDA_ERR_WORKSPACE;
        return cuda_status(kda::launch_prefill_split_noalloc(q, k, v, g, beta, S0, o, S_out,
                                                             cu_seqlens, N, T, H, s));
    }
    // the CUDA-core kernel needs no workspace
    return cuda_status(kda::launch_prefill_simt(q, k, v, g, beta, S0, o, S_out, cu_seqlens, N, T, H,
                                                chunk, dtype == KDA_BF16, s));
}

size_t kda_prefill_workspace_bytes(int N, int64_t T, int H, int dk, int dv, int chunk, int dtype) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return 0;
    if (dk != kda::kDK || dv != kda::kDV || N < 1 || H < 1 || T <= 0 || T >= (int64_t(1) << 31))
        return 0;
    if (dtype != KDA_BF16 || chunk != 64) return 0;
    return kda::prefill_split_workspace_bytes(N, T, H);
}

int kda_prefill_chunked_ws(const void *q, const void *k, const void *v, const float *g,
                           const float *beta, const float *S0, float *o, float *S_out,
                           const int32_t *cu_seqlens, int N, int64_t T, int H, int dk, int dv,
                           int chunk, int dtype, void *workspace, size_t ws_bytes, void *stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (dk != kda::kDK || dv != kda::kDV || N < 1 || H < 1 || T < 0 || T >= (int64_t(1) << 31))
        return KDA_ERR_DIM;
    if ((int64_t)N * H * (kda::kDV / 32) >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (chunk != 16 && chunk != 32 && chunk != 64) return KDA_ERR_CHUNK;
    if (!S_out || !cu_seqlens) return KDA_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !g || !beta || !o)) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, g, beta, S0, o, S_out, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16 && chunk == 64 && T > 0) {
        const size_t need = kda::prefill_split_workspace_bytes(N, T, H);
        if (!workspace || ws_bytes < need) return KDA_ERR_WORKSPACE;
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return KDA_ERR_ALIGN;
        return cuda_status(kda::launch_prefill_split_ws(q, k, v, g, beta, S0, o, S_out, cu_seqlens,
                                                        N, T, H, workspace, s));
    }
    // the CUDA-core kernel needs no workspace
    return cuda_status(kda::launch_prefill_simt(q, k, v, g, beta, S0, o, S_out, cu_seqlens, N, T, H,
                                                chunk, dtype == KDA_BF16, s));
}

int kda_decode_step(const void *q, const void *k, const void *v, const float *g,
                    const float *beta, float *S_inout, float *o, int B, int H, int dk, int dv,
                    int dtype, void *stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (dk != kda::kDK || dv != kda::kDV || B < 0 || H < 1) return KDA_ERR_DIM;
    if ((int64_t)B * H * 2 >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (B == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !S_inout || !o) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, g, beta, S_inout, o};
    for (const void *p : ptrs)
        if (!aligned16(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(kda::launch_decode(q, k, v, g, beta, S_inout, o, B, H, dtype == KDA_BF16, s));
}

int kda_decode_step_pool(const void *q, const void *k, const void *v, const float *g,
                         const float *beta, void *S_pool, int state_dtype,
                         const int32_t *state_indices, int P, float *o, int B, int H, int dk,
                         int dv, int dtype, void *stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (state_dtype != KDA_BF16 && state_dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (dk != kda::kDK || dv != kda::kDV || B < 0 || H < 1 || P < 0) return KDA_ERR_DIM;
    if ((int64_t)B * H * 2 >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (!state_indices && P < B) return KDA_ERR_DIM;
    if (B == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !S_pool || !o) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, g, beta, S_pool, o, state_indices};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(kda::launch_decode_pool(q, k, v, g, beta, S_pool, state_dtype == KDA_BF16,
                                               state_indices, P, o, B, H, dtype == KDA_BF16, s));
}

int kda_conv_prologue(const void *xq, const void *xk, const void *xv, const float *conv_w,
                      const void *conv_in, void *conv_out, void *q, void *k, void *v,
                      const int32_t *cu_seqlens, int N, int64_t T, int H, int d, float q_scale,
                      float eps, void *stream) {
    if (d != kda::kDK || N < 1 || H < 1 || T < 0 || T >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (!(eps >= 0.f) || !(q_scale == q_scale) || q_scale - q_scale != 0.f) return KDA_ERR_VALUE;
    if (!cu_seqlens) return KDA_ERR_NULL;
    if (T > 0 && (!xq || !xk || !xv || !conv_w || !q || !k || !v)) return KDA_ERR_NULL;
    if (conv_in && conv_in == conv_out) return KDA_ERR_VALUE;
    const void *ptrs[] = {xq, xk, xv, conv_w, conv_in, conv_out, q, k, v, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    if (T == 0 && !conv_out) return KDA_OK;
    return cuda_status(kda::launch_conv_prologue(xq, xk, xv, conv_w, conv_in, conv_out, q, k, v,
                                                 cu_seqlens, N, T, H, q_scale, eps,
                                                 static_cast<cudaStream_t>(stream)));
}

int kda_prefill_chunked_gated(const void *q, const void *k, const void *v, const float *g,
                              const float *beta, const float *S0, const void *gate,
                              const float *norm_w, float eps, float *out, float *S_out,
                              const int32_t *cu_seqlens, int N, int64_t T, int H, int dk, int dv,
                              int chunk, int dtype, void *stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (dk != kda::kDK || dv != kda::kDV || N < 1 || H < 1 || T < 0 || T >= (int64_t(1) << 31))
        return KDA_ERR_DIM;
    if ((int64_t)N * H * (kda::kDV / 32) >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (chunk != 16 && chunk != 32 && chunk != 64) return KDA_ERR_CHUNK;
    if (!(eps >= 0.f)) return KDA_ERR_VALUE;
    if (!S_out || !cu_seqlens) return KDA_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !g || !beta || !gate || !norm_w || !out)) return KDA_ERR_NULL;
    const void *ptrs[] = {q, k, v, g, beta, S0, gate, norm_w, out, S_out, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16 && chunk == 64 && T > 0) {
        const cudaError_t e = kda::launch_prefill_split_gated(q, k, v, g, beta, S0, gate, norm_w, eps,
                                                              out, S_out, cu_seqlens, N, T, H, s);
        return e == cudaErrorMemoryAllocation ? KDA_ERR_WORKSPACE : cuda_status(e);
    }
    // CUDA-core prefill into `out`, then the gated norm in place
    cudaError_t e = kda::launch_prefill_simt(q, k, v, g, beta, S0, out, S_out, cu_seqlens, N, T, H,
                                             chunk, dtype == KDA_BF16, s);
    if (e == cudaSuccess) e = kda::launch_gated_norm(out, gate, norm_w, eps, T * H, s);
    return cuda_status(e);
}

int kda_layer_prefill(const void *xq, const void *xk, const void *xv, const float *conv_w,
                      const void *conv_in, void *conv_out, const float *g, const float *beta,
                      const float *S0, const void *gate, const float *norm_w, float q_scale,
                      float l2_eps, float norm_eps, float *out, float *S_out,
                      const int32_t *cu_seqlens, int N, int64_t T, int H, int dk, int dv,
                      void *stream) {
    if (dk != kda::kDK || dv != kda::kDV || N < 1 || H < 1 || T < 0 || T >= (int64_t(1) << 31))
        return KDA_ERR_DIM;
    if ((int64_t)N * H * (kda::kDV / 32) >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (!(l2_eps >= 0.f) || !(norm_eps >= 0.f) || !(q_scale == q_scale) || q_scale - q_scale != 0.f)
        return KDA_ERR_VALUE;
    if (conv_in && conv_in == conv_out) return KDA_ERR_VALUE;
    if (!S_out || !cu_seqlens) return KDA_ERR_NULL;
    if (T > 0 && (!xq || !xk || !xv || !conv_w || !g || !beta || !gate || !norm_w || !out))
        return KDA_ERR_NULL;
    const void *ptrs[] = {xq, xk, xv, conv_w, conv_in, conv_out, g, beta, S0, gate, norm_w, out,
                          S_out, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // every sequence empty: windows and states pass through
        cudaError_t e = cudaSuccess;
        if (conv_out)
            e = kda::launch_conv_prologue(xq, xk, xv, conv_w, conv_in, conv_out, nullptr, nullptr,
                                          nullptr, cu_seqlens, N, T, H, q_scale, l2_eps, s);
        if (e == cudaSuccess)
            e = kda::launch_prefill_simt(nullptr, nullptr, nullptr, g, beta, S0, out, S_out,
                                         cu_seqlens, N, T, H, 64, true, s);
        return cuda_status(e);
    }
    const cudaError_t e = kda::launch_prefill_layer(xq, xk, xv, conv_w, conv_in, conv_out, g, beta,
                                                    S0, gate, norm_w, q_scale, l2_eps, norm_eps,
                                                    out, S_out, cu_seqlens, N, T, H, s);
    return e == cudaErrorMemoryAllocation ? KDA_ERR_WORKSPACE : cuda_status(e);
}

int kda_decode_layer_step(const void *xq, const void *xk, const void *xv, const float *conv_w,
                          void *conv_pool, const float *g, const float *beta, const void *gate,
                          const float *norm_w, void *S_pool, int state_dtype,
                          const int32_t *state_indices, int P, float *out, int B, int H, int dk,
                          int dv, float q_scale, float l2_eps, float norm_eps, void *stream) {
    if (state_dtype != KDA_BF16 && state_dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (dk != kda::kDK || dv != kda::kDV || B < 0 || H < 1 || P < 0) return KDA_ERR_DIM;
    if ((int64_t)B * H >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (!state_indices && P < B) return KDA_ERR_DIM;
    if (!(l2_eps >= 0.f) || !(norm_eps >= 0.f) || !(q_scale == q_scale) || q_scale - q_scale != 0.f)
        return KDA_ERR_VALUE;
    if (B == 0) return KDA_OK;
    if (!xq || !xk || !xv || !conv_w || !conv_pool || !g || !beta || !gate || !norm_w || !S_pool || !out)
        return KDA_ERR_NULL;
    const void *ptrs[] = {xq, xk, xv, conv_w, conv_pool, g, beta, gate, norm_w, S_pool, state_indices, out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_decode_layer(xq, xk, xv, conv_w, conv_pool, g, beta, gate, norm_w,
                                                S_pool, state_dtype == KDA_BF16, state_indices, P,
                                                out, B, H, q_scale, l2_eps, norm_eps,
                                                static_cast<cudaStream_t>(stream)));
}

int kda_latent_append(const void *x, void *cache, const int32_t *block_table, const int32_t *seq_lens,
                      const int32_t *cu_seqlens, const float *norm_w, float eps, int N, int64_t T,
                      int64_t P, int page, int max_pages, int d_latent, int d_pe, void *stream) {
    const int d = latent_cache_dims(N, T, P, page, max_pages, d_latent, d_pe);
    if (d != KDA_OK) return d;
    if (!cu_seqlens && T != N) return KDA_ERR_DIM;
    if (!(eps >= 0.f)) return KDA_ERR_VALUE;
    if (T == 0) return KDA_OK;
    if (!x || !cache || !block_table || !seq_lens) return KDA_ERR_NULL;
    const void *ptrs[] = {x, cache, block_table, seq_lens, cu_seqlens, norm_w};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent_append(x, cache, block_table, seq_lens, cu_seqlens, norm_w,
                                                 eps, N, T, P, page, max_pages,
                                                 static_cast<cudaStream_t>(stream)));
}

int kda_latent_gather(const void *cache, const int32_t *block_table, const int32_t *cu_seqlens,
                      void *out, int N, int64_t T, int64_t P, int page, int max_pages, int d_latent,
                      int d_pe, void *stream) {
    const int d = latent_cache_dims(N, T, P, page, max_pages, d_latent, d_pe);
    if (d != KDA_OK) return d;
    if (T == 0) return KDA_OK;
    if (!cache || !block_table || !cu_seqlens || !out) return KDA_ERR_NULL;
    const void *ptrs[] = {cache, block_table, cu_seqlens, out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent_gather(cache, block_table, cu_seqlens, out, N, T, P, page,
                                                 max_pages, static_cast<cudaStream_t>(stream)));
}

size_t kda_latent_decode_workspace_bytes(int N, int64_t T, int H, int d_latent, int d_pe) {
    if (d_latent != kda::kLatentDim || d_pe != kda::kLatentPeDim || N < 1 || T < 1 || H < 1 ||
        !rows_in_32_bits(T, H))
        return 0;
    return kda::latent_decode_workspace_bytes(N, T, H);
}

int kda_latent_decode(const void *q, const void *cache, const int32_t *block_table,
                      const int32_t *seq_lens, const int32_t *cu_seqlens, float scale, void *o,
                      float *lse, int N, int64_t T, int H, int64_t P, int page, int max_pages,
                      int d_latent, int d_pe, void *workspace, size_t ws_bytes, void *stream) {
    const int d = latent_cache_dims(N, T, P, page, max_pages, d_latent, d_pe);
    if (d != KDA_OK) return d;
    if (H < 1 || !rows_in_32_bits(T, H) || (!cu_seqlens && T != N)) return KDA_ERR_DIM;
    if (!(scale > 0.f) || scale - scale != 0.f) return KDA_ERR_VALUE;
    if (T == 0) return KDA_OK;
    if (!q || !cache || !block_table || !seq_lens || !o) return KDA_ERR_NULL;
    const void *ptrs[] = {q, cache, block_table, seq_lens, cu_seqlens, o, lse};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    const size_t need = kda::latent_decode_workspace_bytes(N, T, H);
    if (need > 0 && (!workspace || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent_decode(q, cache, block_table, seq_lens, cu_seqlens, scale, o,
                                                 lse, N, T, H, P, page, max_pages, workspace,
                                                 static_cast<cudaStream_t>(stream)));
}

size_t kda_latent_prefill_workspace_bytes(int N, int64_t Tq, int64_t Tk, int H, int d_nope, int d_pe, int dv) {
    if (d_nope != kda::kDK || d_pe != kda::kLatentPeDim || dv != kda::kDV || N < 1 || H < 1 || Tq < 1 || Tk < 0 ||
        !rows_in_32_bits(Tq, H) || !rows_in_32_bits(Tk, H))
        return 0;
    return kda::latent_prefill_workspace_bytes(N, Tq, Tk, H);
}

int kda_latent_prefill(const void *q, const void *kv, const void *k_pe, int64_t k_pe_stride,
                       const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, float scale,
                       int causal, void *o, float *lse, int N, int64_t Tq, int64_t Tk, int H,
                       int d_nope, int d_pe, int dv, void *workspace, size_t ws_bytes, void *stream) {
    if (d_nope != kda::kDK || d_pe != kda::kLatentPeDim || dv != kda::kDV) return KDA_ERR_DIM;
    if (N < 1 || H < 1 || Tq < 0 || Tk < 0 || !rows_in_32_bits(Tq, H) || !rows_in_32_bits(Tk, H))
        return KDA_ERR_DIM;
    if (k_pe_stride < d_pe || k_pe_stride % 8 != 0 || k_pe_stride >= (int64_t(1) << 31)) return KDA_ERR_DIM;
    if (!(scale > 0.f) || scale - scale != 0.f || (causal != 0 && causal != 1)) return KDA_ERR_VALUE;
    if (Tq == 0) return KDA_OK;
    if (!q || !cu_seqlens_q || !cu_seqlens_k || !o) return KDA_ERR_NULL;
    if (Tk > 0 && (!kv || !k_pe)) return KDA_ERR_NULL;
    const void *ptrs[] = {q, kv, k_pe, cu_seqlens_q, cu_seqlens_k, o, lse};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    const size_t need = kda::latent_prefill_workspace_bytes(N, Tq, Tk, H);
    if (need > 0 && (!workspace || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent_prefill(q, kv, k_pe, k_pe_stride, cu_seqlens_q, cu_seqlens_k,
                                                  scale, causal != 0, o, lse, N, Tq, Tk, H, workspace,
                                                  static_cast<cudaStream_t>(stream)));
}

int kda_latent_rotate(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
                      int64_t out_token_stride, int64_t out_head_stride, const int64_t *turns,
                      const int32_t *seq_lens, const int32_t *cu_seqlens, float amplitude, int layout,
                      int inverse, int N, int64_t T, int H, int d, int dtype, void *stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (N < 1 || T < 0 || H < 1 || H > (1 << 24) || !rows_in_32_bits(T, H)) return KDA_ERR_DIM;
    if (d < 16 || d > 256 || d % 16 != 0 || (!cu_seqlens && T != N)) return KDA_ERR_DIM;
    const int64_t e = dtype == KDA_BF16 ? 2 : 4;
    if (!row_strides(x_token_stride, x_head_stride, T, H, d, e) ||
        !row_strides(out_token_stride, out_head_stride, T, H, d, e))
        return KDA_ERR_DIM;
    // rows of x may be the same ones (broadcast), rows of out are written once
    if ((T > 1 && out_token_stride < d) || (H > 1 && out_head_stride < d)) return KDA_ERR_DIM;
    if (T > 1 && H > 1) {                     // the tokens' heads apart, or the heads' tokens
        const bool by_token = out_token_stride >= out_head_stride;
        const int64_t outer = by_token ? out_token_stride : out_head_stride;
        const int64_t inner = by_token ? out_head_stride : out_token_stride;
        if (outer < inner * ((by_token ? H : T) - 1) + d) return KDA_ERR_DIM;
    }
    // in place: each row where it was
    if (x == out && ((T > 1 && x_token_stride != out_token_stride) || (H > 1 && x_head_stride != out_head_stride)))
        return KDA_ERR_VALUE;
    const int r = rotation_status(amplitude, layout);
    if (r != KDA_OK) return r;
    if (inverse != 0 && inverse != 1) return KDA_ERR_VALUE;
    if (T == 0) return KDA_OK;
    if (!x || !out || !turns || !seq_lens) return KDA_ERR_NULL;
    const void *ptrs[] = {x, out, turns, seq_lens, cu_seqlens};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent_rotate(
        x, x_token_stride, x_head_stride, out, out_token_stride, out_head_stride,
        kda::Rotation{turns, amplitude, layout == KDA_ROTARY_INTERLEAVED}, inverse != 0, seq_lens, cu_seqlens, N, T, H, d,
        dtype == KDA_BF16, static_cast<cudaStream_t>(stream)));
}

int kda_latent_append_rotated(const void *x, void *cache, const int32_t *block_table,
                              const int32_t *seq_lens, const int32_t *cu_seqlens, const float *norm_w,
                              float eps, const int64_t *turns, float amplitude, int layout, int N,
                              int64_t T, int64_t P, int page, int max_pages, int d_latent, int d_pe,
                              void *stream) {
    const int d = latent_cache_dims(N, T, P, page, max_pages, d_latent, d_pe);
    if (d != KDA_OK) return d;
    if (!cu_seqlens && T != N) return KDA_ERR_DIM;
    if (!(eps >= 0.f)) return KDA_ERR_VALUE;
    const int r = rotation_status(amplitude, layout);
    if (r != KDA_OK) return r;
    if (T == 0) return KDA_OK;
    if (!x || !cache || !block_table || !seq_lens || !turns) return KDA_ERR_NULL;
    const void *ptrs[] = {x, cache, block_table, seq_lens, cu_seqlens, norm_w, turns};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent_append_rotated(
        x, cache, block_table, seq_lens, cu_seqlens, norm_w, eps,
        kda::Rotation{turns, amplitude, layout == KDA_ROTARY_INTERLEAVED}, N, T, P, page, max_pages,
        static_cast<cudaStream_t>(stream)));
}

int kda_latent4_append(const void *x, void *cache, const int32_t *block_table, const int32_t *seq_lens,
                       const int32_t *cu_seqlens, const float *norm_w, float eps, const int64_t *turns,
                       float amplitude, int layout, int exponent, int N, int64_t T, int64_t P, int page,
                       int max_pages, int d_latent, int d_pe, void *stream) {
    const int d = latent_cache_dims(N, T, P, page, max_pages, d_latent, d_pe);
    if (d != KDA_OK) return d;
    if (!cu_seqlens && T != N) return KDA_ERR_DIM;
    if (!(eps >= 0.f)) return KDA_ERR_VALUE;
    const int r = rotation_status(amplitude, layout);
    if (r != KDA_OK) return r;
    if (exponent_status(exponent) != KDA_OK) return KDA_ERR_VALUE;
    if (T == 0) return KDA_OK;
    if (!x || !cache || !block_table || !seq_lens) return KDA_ERR_NULL;
    const void *ptrs[] = {x, cache, block_table, seq_lens, cu_seqlens, norm_w, turns};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    if (!aligned32(cache)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent4_append(
        x, cache, block_table, seq_lens, cu_seqlens, norm_w, eps,
        kda::Rotation{turns, amplitude, layout == KDA_ROTARY_INTERLEAVED}, exponent, N, T, P, page, max_pages,
        static_cast<cudaStream_t>(stream)));
}

int kda_latent4_gather(const void *cache, const int32_t *block_table, const int32_t *cu_seqlens,
                       void *out, int exponent, int N, int64_t T, int64_t P, int page, int max_pages,
                       int d_latent, int d_pe, void *stream) {
    const int d = latent_cache_dims(N, T, P, page, max_pages, d_latent, d_pe);
    if (d != KDA_OK) return d;
    if (exponent_status(exponent) != KDA_OK) return KDA_ERR_VALUE;
    if (T == 0) return KDA_OK;
    if (!cache || !block_table || !cu_seqlens || !out) return KDA_ERR_NULL;
    const void *ptrs[] = {cache, block_table, cu_seqlens, out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return KDA_ERR_ALIGN;
    if (!aligned32(cache)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent4_gather(cache, block_table, cu_seqlens, out, exponent, N, T, P, page,
                                                  max_pages, static_cast<cudaStream_t>(stream)));
}

size_t kda_latent4_decode_workspace_bytes(int N, int64_t T, int H, int d_latent, int d_pe) {
    if (d_latent != kda::kLatentDim || d_pe != kda::kLatentPeDim || N < 1 || T < 1 || H < 1 ||
        !rows_in_32_bits(T, H))
        return 0;
    return kda::latent4_decode_workspace_bytes(N, T, H);
}

int kda_latent4_decode(const void *q, const void *cache, const int32_t *block_table,
                       const int32_t *seq_lens, const int32_t *cu_seqlens, float scale, int exponent,
                       void *o, float *lse, int N, int64_t T, int H, int64_t P, int page, int max_pages,
                       int d_latent, int d_pe, void *workspace, size_t ws_bytes, void *stream) {
    const int d = latent_cache_dims(N, T, P, page, max_pages, d_latent, d_pe);
    if (d != KDA_OK) return d;
    if (H < 1 || !rows_in_32_bits(T, H) || (!cu_seqlens && T != N)) return KDA_ERR_DIM;
    if (!(scale > 0.f) || scale - scale != 0.f || exponent_status(exponent) != KDA_OK) return KDA_ERR_VALUE;
    if (T == 0) return KDA_OK;
    if (!q || !cache || !block_table || !seq_lens || !o) return KDA_ERR_NULL;
    const void *ptrs[] = {q, cache, block_table, seq_lens, cu_seqlens, o, lse};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_ALIGN;
    if (!aligned32(cache)) return KDA_ERR_ALIGN;
    const size_t need = kda::latent4_decode_workspace_bytes(N, T, H);
    if (need > 0 && (!workspace || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent4_decode(q, cache, block_table, seq_lens, cu_seqlens, scale, exponent, o,
                                                  lse, N, T, H, P, page, max_pages, workspace,
                                                  static_cast<cudaStream_t>(stream)));
}

int kda_workspace_release(void) { return cuda_status(kda::release_workspace_pool()); }

int kda_device_error(unsigned int *code, int reset) {
    if (!code) return KDA_ERR_NULL;
    cudaError_t (*const words[])(unsigned int *, bool) = {
        kda::read_device_error, kda::read_decode_error,         kda::read_layer_error,
        kda::read_simt_error,   kda::read_latent_error,         kda::read_latent_prefill_error,
        kda::read_latent_decode_error, kda::read_rotary_error,  kda::read_latent4_error,
        kda::read_latent4_decode_error};
    cudaError_t first = cudaSuccess;
    *code = 0;
    for (const auto read : words) {
        unsigned int w = 0;
        const cudaError_t e = read(&w, reset != 0);
        *code |= w;
        if (first == cudaSuccess) first = e;
    }
    if (first != cudaSuccess) return cuda_status(first);
    return KDA_OK;
}

#ifdef KDA_DEBUG
// Not part of the ABI: lets a test make a bounded wait of the decode (prefill)
// kernel's next calls run out; 0xffffffff ends that.
int kda_debug_latent_leave_out(unsigned int decode_tile, unsigned int prefill_tile) {
    const cudaError_t e = kda::latent_decode_leave_out(decode_tile);
    return cuda_status(e == cudaSuccess ? kda::latent_prefill_leave_out(prefill_tile) : e);
}
// The same for the decode kernel of the 4-bit cache.
int kda_debug_latent4_leave_out(unsigned int tile) { return cuda_status(kda::latent4_decode_leave_out(tile)); }
#endif

}  // extern "C"
