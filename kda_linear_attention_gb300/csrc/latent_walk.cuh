// What the absorbed decode kernels share: how the work of a batch is cut into
// units of (sequence, row tile, 128 positions) and dealt out to the CTAs, the
// walk over a CTA's units, and the kernel that joins the pieces of row tiles
// that several CTAs had.
#pragma once

#include <algorithm>

#include "latent_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kTile = 128;                // positions a unit
// Units that a row tile counts beside its tiles of positions, in front of them
// (queries, first scores, output).  24 sequences of 100-2,100 tokens with
// drafts: 26.0 us without, 24.3 with one, 24.5 with two; 64 of 2,000-4,096 at
// 96 heads: 75, 73, 74; 128 of 8,000-8,192 at 64 heads: 207, 208, 208.
constexpr int kExtra = 1;
constexpr int kMaxCtas = 160;             // grid bound (one CTA an SM; 152 SMs)
constexpr int kMaxSide = 8;               // row tiles of a token that CTAs take side by side

// What a CTA leaves for the joining kernel: the row tile that starts in its
// units and goes on behind them.
struct Split {
    int32_t row;                          // first row (flat over [T * H])
    int32_t rows;                         // rows of the tile; 0: nothing
    int32_t pieces;                       // of it: here and in the CTAs `side` further on each
    int32_t blind;                        // its first rows, which see nothing
};

// The batch of a call.
struct Batch {
    PagedRows pages;
    const int32_t *seq_lens, *cu;
    int N, T, H;
    int side;                             // CTAs side by side: row tiles of a token (one token a sequence)
};

// A sequence as the kernel sees it (clamped to what its buffers hold).
struct Seq {
    int row0, rows;                       // flat rows over [T * H], of this sequence
    int first;                            // positions its first new token sees (may be <= 0)
    int len, units, row_tiles;            // units: of each of its row tiles
};

// A CTA's first unit and how many it has (shared memory).
struct Begin {
    int b0, j0, t0;                       // first unit
    Seq seq0;                             // its sequence
    long long scan[32];
    long long start, units, each;         // this CTA's first unit and units; a group's units
};

// What is wrong with it raises bit 0 of *error, where that is given.
template <int NR>
__device__ __forceinline__ Seq get_seq(const Batch &a, int b, unsigned int *error) {
    const int j = blockIdx.x % a.side;    // with side > 1 every CTA knows its row tile only
    Seq s;
    int t0 = b, n = 1;
    bool bad = false;
    if (a.cu) {
        t0 = a.cu[b];
        const int t1 = a.cu[b + 1];
        bad = t0 < 0 || t1 < t0 || t1 > a.T;
        n = bad ? 0 : t1 - t0;
        if (bad) t0 = 0;
    }
    int L = a.seq_lens[b];
    const int most = a.pages.max_len();
    if (L < 0 || L > most) {
        bad = true;
        L = max(0, min(L, most));
    }
    if (bad && error) atomicOr(error, kErrWait);
    s.row0 = t0 * a.H + j * NR;
    s.rows = a.side > 1 ? min(NR, a.H - j * NR) : n * a.H;
    s.first = L - n + 1;
    s.len = L;
    s.units = max(1, (L + kTile - 1) / kTile) + kExtra;
    s.row_tiles = (s.rows + NR - 1) / NR;
    return s;
}

// One row tile over a range of positions.
struct Item {
    int b, row, rows;                     // sequence, first flat row, rows
    int tile, n;                          // first tile of positions, tiles with anything to see
    int len;                              // the sequence's length
    int first_tok, row_in_seq;            // positions its first new token sees; row - row0
    bool head, tail;                      // holds the row tile's first / last tile of positions
    long long unit;                       // the unit of its first tile
    int tiles;                            // tiles of the whole row tile
};

// Walks a CTA's units row tile by row tile; every role takes the same walk.
template <int NR>
struct Walk {
    int b, j, t;
    long long left, u;
    Seq s;
    __device__ __forceinline__ Walk(const Batch &a, const Begin &m)
        : b(m.b0), j(m.j0), t(m.t0), left(m.units), u(m.start) {
        if (left > 0) s = m.seq0;
    }
    __device__ __forceinline__ bool next(const Batch &a, Item &it) {
        int from, to;                     // tiles of positions
        do {
            if (left <= 0) return false;
            while (j >= s.row_tiles) {    // units are left, so a sequence with rows follows
                if (++b >= a.N) { left = 0; return false; }
                s = get_seq<NR>(a, b, nullptr);
                j = t = 0;
            }
            const int units = (int)min((long long)(s.units - t), left);
            from = max(0, t - kExtra);
            to = max(0, t + units - kExtra);
            it.unit = u - t + kExtra;
            it.row_in_seq = j * NR;
            left -= units;
            u += units;
            t = 0;
            ++j;
        } while (to <= from);             // none of its tiles is here
        it.b = b;
        it.row = s.row0 + it.row_in_seq;
        it.rows = min(NR, s.rows - it.row_in_seq);
        it.len = s.len;
        it.first_tok = s.first;
        it.head = from == 0;
        it.tail = to == s.units - kExtra;
        it.tile = from;
        it.tiles = s.units - kExtra;
        // the last row sees the most positions
        const int most = min(s.len, s.first + (it.row_in_seq + it.rows - 1) / a.H);
        it.n = max(0, min(to, (max(0, most) + kTile - 1) / kTile) - from);
        return true;
    }
};

// This CTA's units: a block-wide scan of the sequences' units, by all THREADS
// threads; *m holds them after the next block barrier.
template <int NR, int THREADS>
__device__ __forceinline__ void find_units(const Batch &a, Begin *m, unsigned int *error) {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, cta = blockIdx.x;
    const int G = gridDim.x / a.side, group = cta / a.side;   // groups of CTAs side by side
    if (t == 0) m->b0 = m->j0 = m->t0 = 0;
    const int per = (a.N + THREADS - 1) / THREADS;
    const int b_lo = min(a.N, t * per), b_hi = min(a.N, b_lo + per);
    long long mine = 0;
    Seq s;                                         // the only one where there are few
    for (int b = b_lo; b < b_hi; ++b) {
        s = get_seq<NR>(a, b, cta == 0 ? error : nullptr);   // CTA 0 flags what is wrong with a sequence
        mine += (long long)s.units * s.row_tiles;
    }
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) m->scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += m->scan[w];
        total += m->scan[w];
    }
    // as many units for each group as the one with the most must have: fewer groups, and fewer
    // pieces, where that leaves some without
    const long long each = max(1LL, (total + G - 1) / G);
    const long long u0 = min(total, group * each), u1 = group < G ? min(total, u0 + each) : u0;
    if (t == 0) {
        m->units = u1 - u0;
        m->start = u0;
        m->each = each;
    }
    if (u1 > u0 && u0 >= before && u0 < before + mine) {
        for (int b = b_lo; b < b_hi; ++b) {
            if (per > 1) s = get_seq<NR>(a, b, nullptr);
            const long long n = (long long)s.units * s.row_tiles;
            if (u0 < before + n) {
                m->b0 = b;
                m->seq0 = s;
                m->j0 = (int)((u0 - before) / s.units);
                m->t0 = (int)((u0 - before) % s.units);
                break;
            }
            before += n;
        }
    }
}

// Sum (or maximum) over the 32 lanes of each of NC values: lane l of the
// result holds value l (l < NC), for NC a multiple of 8 up to 32.
template <int NC, bool MAX>
__device__ __forceinline__ float lanes_reduce(float (&v)[NC], int lane) {
    float r = 0.f;
#pragma unroll
    for (int c = 0; c < NC; c += 8) {
        // butterfly over 8 columns: after 3 halvings a lane holds one column
        // over 4-lane strided groups, then two more exchanges finish it
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = v[c + i];
#pragma unroll
        for (int h = 4; h > 0; h >>= 1) {
            const bool up = lane & h;
#pragma unroll
            for (int i = 0; i < h; ++i) {
                const float keep = up ? w[i + h] : w[i], give = up ? w[i] : w[i + h];
                const float got = __shfl_xor_sync(0xffffffffu, give, h);
                w[i] = MAX ? fmaxf(keep, got) : keep + got;
            }
        }
        // lane l holds column c + (l & 7) over the lanes with its low bits
#pragma unroll
        for (int h = 8; h < 32; h <<= 1) {
            const float got = __shfl_xor_sync(0xffffffffu, w[0], h);
            w[0] = MAX ? fmaxf(w[0], got) : w[0] + got;
        }
        if ((lane >> 3) == (c >> 3)) r = w[0];
    }
    return r;
}

// Joins the pieces of the row tiles that start in one CTA and go on behind
// it: o = sum_k 2^(lse_k - lse) o_k, in the order of the positions.  Every
// block lists all such tiles (at most one a CTA) and takes every gridDim-th
// unit of them: eight slices of rows, a warp each, or one row's slice of a
// tile with many pieces and few rows, which the block's warps share and whose
// warps' sums are added in order.
// Bound by latency and by its own instructions (100 to 400 a slice); the
// pieces come from L2, where the first kernel has just left them.  So a warp
// asks for its pieces before it has their weights, and few pieces make a wide
// slice, whose weights cost less, many a narrow one, of which there are more
// at the same time.  Measured, in a graph, against whole rows, two pieces at a
// time behind their weights: one sequence of 1,000 tokens at 16 heads 10.7 us
// a call (12.8), 24 of 100-2,100 with drafts 22.2 (23.8), 16 of 8,192 at 64
// heads 47.2 (51.5), 131,072 and 100,001 at 32 heads 58.7 (61.7), 64 of
// 2,000-4,096 at 96 heads 73.9 (74.4); 24 of 3,000 at 128 heads 44.2 (42.5).
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = 32 * kJoinWarps;
// Pieces a warp takes by itself: in slices of 256 channels, in slices of 128,
// in slices of 128 where the rows are many beside them.  (Wide slices up to 4
// pieces: 24 of 3,000 at 128 heads 43.6 us, 64 of 2,000-4,096 at 96 74.2; a
// block a slice from 9 on whatever the rows: 16 of 8,192 at 64 heads 60.)
constexpr int kJoinWide = 3, kJoinNarrow = 8, kJoinMost = 32;
static_assert(kJoinThreads >= kMaxCtas, "a thread a record");

struct JoinArgs {
    const Split *split;
    const float *ws_lse, *ws_o;
    __nv_bfloat16 *o;
    float *lse;
    int NR, ctas, side;
};

// Weights of a row's pieces, in each group of L lanes a lane's of piece L e +
// lane, from their log2-sum-exp; returns the row's.  NaN in a piece makes all of
// them NaN; where none has any weight they are 0 for a blind row and NaN (0 / 0)
// for one that sees positions, whose scores are all -inf; ln 0 = -inf for both.
template <int L, int E>
__device__ __forceinline__ float join_weights(float (&v)[E], bool blind) {
    float mx = -kHuge, sum = 0.f;             // finite, so that no weight is -inf - -inf
#pragma unroll
    for (int e = 0; e < E; ++e) mx = fmaxf(mx, v[e]);
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
#pragma unroll
    for (int e = 0; e < E; ++e) {
        v[e] = ex2_approx(v[e] - mx);
        sum += v[e];
    }
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float inv = blind ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= inv;
    return mx + log2f(sum);
}
__device__ __forceinline__ void add_scaled(float4 &acc, float w, const float4 &x) {
    acc.x = fmaf(w, x.x, acc.x);
    acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z);
    acc.w = fmaf(w, x.w, acc.w);
}

__device__ __forceinline__ bool join_alone(int n, int NR) { return n <= kJoinNarrow || (n <= kJoinMost && NR > 2 * n); }

// A warp joins slice `sl` (128 W channels) of row r of CTA c's tile of up to N pieces, K of them in
// flight together.
template <int N, int K, int W>
__device__ __forceinline__ void join_row(const JoinArgs &a, int c, const Split &sp, int r, int sl, int lane) {
    const int n = sp.pieces;
    // where piece 0 and piece 1 have the row; the further ones lie a stride apart (the workspace has
    // less than 2^25 numbers)
    const int stride = 2 * a.side * a.NR, row0 = (2 * c + 1) * a.NR + r, row1 = 2 * c * a.NR + stride + r;
    constexpr int L = N <= 4 ? 4 : N <= 8 ? 8 : 32;           // lanes that share the weights out
    const int mine = lane % L;
    float v[1] = {mine < n ? a.ws_lse[mine == 0 ? row0 : row1 + (mine - 1) * stride] : -CUDART_INF_F}, lg = 0.f;
    const float4 *const src = reinterpret_cast<const float4 *>(a.ws_o) + 32 * W * sl + lane;
    float4 acc[W];
#pragma unroll
    for (int q = 0; q < W; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < (N > K ? n : 1); k0 += K) {
        float4 x[K][W];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int row = k0 + k == 0 ? row0 : row1 + (k0 + k - 1) * stride;
#pragma unroll
            for (int q = 0; q < W; ++q)
                x[k][q] = k0 + k < n ? src[row * (kLatent / 4) + 32 * q] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (k0 == 0) lg = join_weights<L>(v, r < sp.blind);   // behind the first loads
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float w = __shfl_sync(0xffffffffu, v[0], k0 + k);   // from the n-th on any: x is 0
#pragma unroll
            for (int q = 0; q < W; ++q) add_scaled(acc[q], w, x[k][q]);
        }
    }
    const size_t row = (size_t)sp.row + r;
    uint2 *dst = reinterpret_cast<uint2 *>(a.o + row * kLatent);
#pragma unroll
    for (int q = 0; q < W; ++q)
        dst[32 * (W * sl + q) + lane] = make_uint2(pack_bf2(acc[q].x, acc[q].y), pack_bf2(acc[q].z, acc[q].w));
    if (a.lse && sl == 0 && lane == 0) a.lse[row] = lg * 0.6931471805599453f;
}

__global__ void __launch_bounds__(kJoinThreads, 4)
latent_join_kernel(const JoinArgs a) {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    __shared__ float4 part[kJoinWarps][32];
    __shared__ float weight[kMaxCtas];
    __shared__ Split rec[kMaxCtas];
    __shared__ int upto[kJoinThreads];        // units of the records up to and with this one
    __shared__ int warp_sum[kJoinWarps];
    let_next_begin();
    wait_for_previous();                      // the pieces are written
    {
        Split sp{0, 0, 0, 0};
        if (t < a.ctas) {
            sp = a.split[t];
            rec[t] = sp;
        }
        const int slices = sp.rows * (sp.pieces <= kJoinWide ? 2 : 4);
        int incl = join_alone(sp.pieces, a.NR) ? (slices + kJoinWarps - 1) / kJoinWarps : slices;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += warp_sum[w];
        upto[t] = incl;
        __syncthreads();
    }
    const int units = upto[kJoinThreads - 1];
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        int c = 0, hi = kJoinThreads - 1;         // the first record that reaches past u
        while (c < hi) {
            const int mid = (c + hi) >> 1;
            if (upto[mid] > u) hi = mid;
            else c = mid + 1;
        }
        const Split sp = rec[c];
        const int n = sp.pieces, in = u - (c > 0 ? upto[c - 1] : 0);
        if (join_alone(n, a.NR)) {
            const int i = in * kJoinWarps + warp, per = n <= kJoinWide ? 2 : 4;
            if (i >= sp.rows * per) continue;
            if (n <= kJoinWide) join_row<kJoinWide, kJoinWide, 2>(a, c, sp, i >> 1, i & 1, lane);
            else join_row<kJoinMost, 4, 1>(a, c, sp, i >> 2, i & 3, lane);
            continue;
        }
        // warp w takes the pieces w, w + 8, .. of 128 channels, eight of them at a time
        const int r = in >> 2, sl = in & 3;
        const int stride = 2 * a.side * a.NR, row0 = (2 * c + 1) * a.NR + r, row1 = 2 * c * a.NR + stride + r;
        const float4 *const src = reinterpret_cast<const float4 *>(a.ws_o) + 32 * sl + lane;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float lg = 0.f;
#pragma unroll 1
        for (int k0 = warp; k0 < n; k0 += 8 * kJoinWarps) {
            float4 x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int k = k0 + e * kJoinWarps;
                x[e] = k < n ? src[(k == 0 ? row0 : row1 + (k - 1) * stride) * (kLatent / 4)]
                             : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (k0 == warp) {                 // behind the first loads; every warp has some (n > 8)
                if (warp == 0) {
                    float v[kMaxCtas / 32];
#pragma unroll
                    for (int e = 0; e < kMaxCtas / 32; ++e) {
                        const int k = 32 * e + lane;
                        v[e] = k < n ? a.ws_lse[k == 0 ? row0 : row1 + (k - 1) * stride] : -CUDART_INF_F;
                    }
                    lg = join_weights<32>(v, r < sp.blind);
#pragma unroll
                    for (int e = 0; e < kMaxCtas / 32; ++e) weight[32 * e + lane] = v[e];
                }
                __syncthreads();
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int k = k0 + e * kJoinWarps;
                if (k < n) add_scaled(acc, weight[k], x[e]);
            }
        }
        part[warp][lane] = acc;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w) {
                const float4 y = part[w][lane];
                acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
            }
            const size_t row = (size_t)sp.row + r;
            reinterpret_cast<uint2 *>(a.o + row * kLatent)[32 * sl + lane] =
                make_uint2(pack_bf2(acc.x, acc.y), pack_bf2(acc.z, acc.w));
            if (a.lse && sl == 0 && lane == 0) a.lse[row] = lg * 0.6931471805599453f;
        }
        __syncthreads();
    }
}

// Rows of a tile, in steps of 16 (the products' column step) up to 64.  One
// token a sequence: its H rows in as few tiles as hold them.  More tokens, and
// then ragged ones: a third more than the average sequence's rows, because a
// tile costs little more with more columns (a product step reads a 128-lane
// operand beside them: alone 40 cycles at 32 columns, 48 at 64) and a second
// tile for the longer sequences' last rows costs as much as the first.
int rows_of_tile(int N, int64_t T, int H) {
    const int64_t rows = T == N ? H : (T * H + N - 1) / N * 4 / 3;
    const int64_t tiles = (rows + 63) / 64;
    return (int)std::min<int64_t>(64, std::max<int64_t>(1, ((rows + tiles - 1) / tiles + 15) / 16) * 16);
}

constexpr size_t kSplitBytes = 4096, kLseBytes = 2 * kMaxCtas * 64 * sizeof(float);
static_assert(kSplitBytes >= kMaxCtas * sizeof(Split), "records of the split row tiles");

// Bytes of the split records, the pieces' log2-sum-exp and the pieces.
size_t pieces_bytes(int NR) {
    return kSplitBytes + kLseBytes + (size_t)2 * kMaxCtas * NR * kLatent * sizeof(float);
}

// Row tiles that CTAs take side by side.  One token a sequence and more heads
// than a tile's rows: the row tiles of a sequence are taken by neighbouring
// CTAs at the same time, so that its cached rows come from HBM once.  With
// offsets the host does not know the sequences' row tiles, and a CTA walks them
// one after the other: over the bf16 cache, 64 sequences of 2,000-4,096 tokens
// at 96 heads 75 us without offsets, 91 us with them, at 128 heads 82 and 97.
int tiles_side_by_side(const int32_t *cu, int H, int NR) {
    const int row_tiles = cu ? 1 : (H + NR - 1) / NR;
    return row_tiles <= kMaxSide ? row_tiles : 1;
}

}  // namespace
}  // namespace kda
