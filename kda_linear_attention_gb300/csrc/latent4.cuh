// The 4-bit latent row as the kernels see it: 256 bytes of e2m1 codes, the
// shared part in bf16, 32 e4m3 scales of 16 channels each.  All three parts
// begin at multiples of 32 bytes, so that a row is read in whole sectors.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "latent_common.cuh"

namespace kda {

constexpr int k4Pe = kLatent / 2;                       // byte offset of the shared part
constexpr int k4Scales = k4Pe + 2 * kLatentPeDim;       // ... of the scales
constexpr int k4Groups = kLatent / 16;
static_assert(kLatent4Row == k4Scales + k4Groups && kLatent4Row == 416, "the documented row");

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 h2_of(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// Two codes (a byte, the low half first) as fp16, which holds them exactly.
__device__ __forceinline__ __half2 codes2(uint32_t byte) {
    return __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1));
}
// Two scales (the low byte first) as fp16, exact; NaN stays NaN.
__device__ __forceinline__ __half2 scales2(uint32_t two) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}
// 2^e as fp32, -126 <= e <= 127.
__host__ __device__ __forceinline__ float pow2(int e) {
#ifdef __CUDA_ARCH__
    return __int_as_float((e + 127) << 23);
#else
    float r = 1.f;
    for (; e > 0; --e) r *= 2.f;
    for (; e < 0; ++e) r *= 0.5f;
    return r;
#endif
}

}  // namespace kda
