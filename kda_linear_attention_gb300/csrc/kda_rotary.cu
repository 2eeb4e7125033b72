// Rotary positions on a part of the heads' rows.
//
// A block takes the heads of a few tokens: the tokens' cosines and sines are
// computed once into shared memory (a pair a thread; sincospif is some 40
// instructions, against a handful for the rotation itself), then each thread
// turns two pieces of eight channels at a time, the pairs' two halves
// (KDA_ROTARY_HALF) or 16 channels in a row (KDA_ROTARY_INTERLEAVED).  The
// first pieces are asked for before the angles.
// Bound by HBM: d channels in and out a row.  66,048 tokens of 96 heads, 64 of
// 192 channels of each in bf16: 259 us, 92 % of the measured copy (two units a
// thread, all loaded together: 312 us at two, 374 at four; eight, four together:
// 264; 16: 265).
#include <algorithm>

#include "latent_rows.cuh"

namespace kda {

// Error word of this file's kernels (bit 0: offsets, a length or a position
// out of range).
__device__ unsigned int g_kda_rotary_error = 0;

namespace {

constexpr int kRotateThreads = 256;
constexpr int kMaxTokens = 32;             // of a block
constexpr int kMaxPairs = 2048;            // of a block's tokens: 16 KB
constexpr int kUnits = 8;                  // of a thread, where there are tokens enough
constexpr int kInFlight = 2;               // ... that are loaded together

struct RotateArgs {
    const uint8_t *x;
    uint8_t *out;
    int64_t x_token, x_head, out_token, out_head;   // bytes
    Rotation rot;
    const int32_t *seq_lens, *cu;
    int N, T, H, d, tokens;                // tokens of a block
    bool inverse;
};

// Eight channels as they lie in memory.
template <typename E>
struct Piece {
    uint4 v[sizeof(E) / 2];
    __device__ __forceinline__ void load(const uint8_t *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(E) / 2; ++i) v[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void store(uint8_t *p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(E) / 2; ++i) __stcs(reinterpret_cast<uint4 *>(p) + i, v[i]);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        if constexpr (sizeof(E) == 2) {
            tc::unpack_bf8(v[0], f);
        } else {
            const float *w = reinterpret_cast<const float *>(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = w[i];
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        if constexpr (sizeof(E) == 2) {
            v[0] = tc::pack_bf8(f);
        } else {
            float *w = reinterpret_cast<float *>(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = f[i];
        }
    }
};

template <typename E, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotateThreads)
latent_rotate_kernel(const RotateArgs a) {
    __shared__ float2 angle[kMaxPairs];
    __shared__ bool live[kMaxTokens];
    tc::let_next_begin();
    tc::wait_for_previous();
    check_offsets(a.cu, a.N, a.T, &g_kda_rotary_error);
    const int t0 = blockIdx.x * a.tokens, tokens = min(a.tokens, a.T - t0);
    const int pairs = a.d / 2, per_row = a.d / 16;
    const int units = tokens * a.H * per_row;
    const int gap = (INTERLEAVED ? 8 : a.d / 2) * (int)sizeof(E);   // between a unit's two pieces
    Piece<E> u[kInFlight], v[kInFlight];
    auto place = [&](int unit, int &tok, int &c, int64_t &from, int64_t &to) {
        const int row = unit / per_row;
        c = unit - row * per_row;
        tok = row / a.H;
        const int h = row - tok * a.H;
        const int64_t at = (int64_t)c * (INTERLEAVED ? 16 : 8) * (int)sizeof(E);
        from = (int64_t)(t0 + tok) * a.x_token + h * a.x_head + at;
        to = (int64_t)(t0 + tok) * a.out_token + h * a.out_head + at;
    };
    auto fetch = [&](int first) {
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int unit = first + k * kRotateThreads;
            if (unit >= units) break;
            int tok, c;
            int64_t from, to;
            place(unit, tok, c, from, to);
            u[k].load(a.x + from);
            v[k].load(a.x + from + gap);
        }
    };
    fetch(threadIdx.x);
    for (int i = threadIdx.x; i < tokens * pairs; i += kRotateThreads) {
        const int tok = i / pairs, t = t0 + tok, s = seq_of_token(a.cu, a.N, t);
        long long pos = -1;
        if (s >= 0) {
            const int start = a.cu ? a.cu[s] : s, count = a.cu ? a.cu[s + 1] - start : 1;
            const int len = a.seq_lens[s];
            pos = (long long)len - count + (t - start);
            if (pos < 0) atomicOr(&g_kda_rotary_error, kErrWait);
        }
        if (i == tok * pairs) live[tok] = pos >= 0;
        float2 cs = pos >= 0 ? rotation_of(a.rot, i - tok * pairs, (int)pos) : make_float2(0.f, 0.f);
        if (a.inverse) cs.y = -cs.y;
        angle[i] = cs;
    }
    __syncthreads();
    for (int first = threadIdx.x; first < units; first += kInFlight * kRotateThreads) {
        if (first != threadIdx.x) fetch(first);
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int unit = first + k * kRotateThreads;
            if (unit >= units) break;
            int tok, c;
            int64_t from, to;
            place(unit, tok, c, from, to);
            if (!live[tok]) continue;
            const float2 *cs = angle + tok * pairs + 8 * c;
            float p[8], q[8];
            u[k].get(p);
            v[k].get(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float &x = INTERLEAVED ? (i < 4 ? p[2 * i] : q[2 * i - 8]) : p[i];
                float &y = INTERLEAVED ? (i < 4 ? p[2 * i + 1] : q[2 * i - 7]) : q[i];
                const float2 r = rotated(x, y, cs[i]);
                x = r.x;
                y = r.y;
            }
            u[k].set(p);
            v[k].set(q);
            u[k].store(a.out + to);
            v[k].store(a.out + to + gap);
        }
    }
}

}  // namespace

cudaError_t launch_latent_rotate(const void *x, int64_t x_token, int64_t x_head, void *out, int64_t out_token,
                                 int64_t out_head, const Rotation &rot, bool inverse, const int32_t *seq_lens,
                                 const int32_t *cu, int N, int64_t T, int H, int d, bool bf16,
                                 cudaStream_t stream) {
    const int64_t e = bf16 ? 2 : 4;
    // enough tokens for kUnits a thread, few enough for their angles and for two blocks on each of 152 SMs
    const int64_t units = (int64_t)H * (d / 16);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kUnits * kRotateThreads / units, T / 304));
    const int tokens = (int)std::min<int64_t>(std::min<int64_t>(want, kMaxTokens), kMaxPairs / (d / 2));
    const RotateArgs a{static_cast<const uint8_t *>(x), static_cast<uint8_t *>(out), x_token * e, x_head * e,
                       out_token * e, out_head * e, rot, seq_lens, cu, N, (int)T, H, d, tokens, inverse};
    const unsigned blocks = (unsigned)((T + tokens - 1) / tokens);
    auto kernel = bf16 ? (rot.interleaved ? latent_rotate_kernel<__nv_bfloat16, true> : latent_rotate_kernel<__nv_bfloat16, false>)
                       : (rot.interleaved ? latent_rotate_kernel<float, true> : latent_rotate_kernel<float, false>);
    return tc::launch_early(kernel, blocks, kRotateThreads, 0, stream, a);
}

cudaError_t read_rotary_error(unsigned int *code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kda_rotary_error, sizeof(unsigned int));
    if (e != cudaSuccess || !reset) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kda_rotary_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
