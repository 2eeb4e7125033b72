// Pieces shared by the kernels that write and read cached rows: the offsets'
// check, the latent part's RMS norm, the rotation of the shared part.
#pragma once

#include "latent_tc.cuh"

namespace kda {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// warp_sum of x_l + x_(32 + l) where lane l holds x_2l and x_(2l + 1): the same additions in the same
// order, so the same bits.
__device__ __forceinline__ float warp_sum_of_neighbours(float even, float odd, int lane) {
    const bool up = lane & 16;            // the lower lanes go on with the even ones, the upper with the odd
    float x = (up ? odd : even) + __shfl_xor_sync(0xffffffffu, up ? even : odd, 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Block 0 raises bit 0 of its file's error word for offsets that decrease or leave [0, T] (the rest of
// the kernel stays inside its buffers whatever they are).
__device__ __forceinline__ void check_offsets(const int32_t *cu, int N, int T, unsigned int *error) {
    if (!cu || blockIdx.x != 0) return;
    bool bad = false;
    for (int b = threadIdx.x; b < N; b += blockDim.x) bad |= cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > T;
    if (bad) atomicOr(error, kErrWait);
}

// ---- the RMS norm of a row's latent part, eight channels at a time
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

// ---- rotation
// cos and sin (times the amplitude) of the angle of `pair` at position pos >= 0.
// pos * turns wraps at whole turns, so what is left is the angle's part of a turn
// to 2^-64 of its frequency's rounding; its upper 32 bits, signed, go on in fp32
// (2^-25 of a half turn).
__device__ __forceinline__ float2 rotation_of(const Rotation &rot, int pair, int pos) {
    const uint64_t turn = (uint64_t)pos * (uint64_t)rot.turns[pair];
    const int32_t half_turns = (int32_t)((turn + 0x80000000ull) >> 32);   // in 2^-31 of a half turn
    float s, c;
    sincospif((float)half_turns * 0x1p-31f, &s, &c);
    return make_float2(c * rot.amplitude, s * rot.amplitude);
}
__device__ __forceinline__ float2 rotated(float a, float b, float2 cs) {
    return make_float2(a * cs.x - b * cs.y, b * cs.x + a * cs.y);
}
// The shared part of a row by one warp, a pair a lane (two bf16): read ...
__device__ __forceinline__ uint32_t load_pair(const __nv_bfloat16 *pe, int lane, bool interleaved) {
    if (interleaved) return reinterpret_cast<const uint32_t *>(pe)[lane];
    const uint16_t *h = reinterpret_cast<const uint16_t *>(pe);
    return h[lane] | (uint32_t)h[lane + kLatentPeDim / 2] << 16;
}
// ... turned, with one rounding ...
__device__ __forceinline__ uint32_t turned_pair(uint32_t pair, float2 cs) {
    const float2 v = bf2_to_f2(pair);
    return f2_to_bf2(rotated(v.x, v.y, cs));
}
// ... and written.
__device__ __forceinline__ void store_pair(__nv_bfloat16 *pe, int lane, bool interleaved, uint32_t pair) {
    if (interleaved) {
        reinterpret_cast<uint32_t *>(pe)[lane] = pair;
    } else {
        uint16_t *h = reinterpret_cast<uint16_t *>(pe);
        h[lane] = (uint16_t)pair;
        h[lane + kLatentPeDim / 2] = (uint16_t)(pair >> 16);
    }
}
static_assert(kLatentPeDim == 64, "a pair a lane");

// Where a new token's row goes: its position and cache row; a row of -1 for a
// token that no sequence holds, and for a bad place, whose bit it raises.
struct NewRow {
    int pos;
    int64_t row;
};
__device__ __forceinline__ NewRow new_row(const PagedRows &pages, const int32_t *seq_lens, const int32_t *cu, int N,
                                          int t, int lane, unsigned int *error) {
    const int s = seq_of_token(cu, N, t);
    if (s < 0) return NewRow{0, -1};       // behind the last sequence
    const int start = cu ? cu[s] : s, count = cu ? cu[s + 1] - start : 1;
    const long long pos = (long long)seq_lens[s] - count + (t - start);
    if (pos < 0 || pos >= pages.max_len()) {
        if (lane == 0) atomicOr(error, kErrWait);
        return NewRow{0, -1};
    }
    const int64_t row = pages.row(s, (int)pos);
    if (row < 0 && lane == 0) atomicOr(error, kErrSlot);
    return NewRow{(int)pos, row};
}

}  // namespace kda
