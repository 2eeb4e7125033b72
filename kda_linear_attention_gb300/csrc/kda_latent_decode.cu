// Absorbed latent attention of one or a few new tokens a sequence over the
// paged cache, on the tensor cores.
//
// A sequence's n new tokens and H heads are n H rows x [576] that attend to
// the same cached rows [c | r] (512 + 64), so a tile of 128 positions is read
// once for up to 64 of them.  Both products run with the positions or the
// latent channels on the 128 TMEM lanes and the rows as columns, so a few
// rows cost a few columns:
//   S^T [128 positions x rows]   = K [128 x 576] X^T           (36 K-steps)
//   O^T [512 x rows]            += c^T [512 x 128] P^T         (4 blocks of 128 channels, 8 K-steps)
// K's tile is both products' A operand, K-major for the first, MN-major for
// the second.  P = exp2(S scale log2 e - m) in bf16 (fp32 sums of the
// unrounded values): the product takes bf16 operands, and P's rounding, 2^-8 of
// each probability at most and independent of the others', is of the kind that
// the bf16 output has anyway (against 64 bits 1.7e-3 to 2.0e-3 in the 2-norm; the
// output's rounding alone makes 1.6e-3 to 1.7e-3).  m is a row's running maximum,
// moved only when a score passes it by more than 8 (a factor 256, which fp32
// sums and bf16 probabilities hold without loss); then O^T and the sums are
// rescaled in TMEM and registers.
//
// Work is cut in units of (sequence, row tile, 128 positions), and one more a
// row tile for what it costs beside them; with W units on G CTAs (one an SM)
// each takes the next ceil(W / G), whatever the lengths are.  (The row tiles
// of one token of many heads are taken side by side, by groups of CTAs that
// share the units' numbering, where the call gives no offsets.)  A CTA's first
// and last row tile may be pieces of longer ones: pieces are written normalised
// in fp32 with their log2-sum-exp into the workspace, and a second kernel joins
// them in the order of the positions (no atomics: the same bits every time).
//
// Roles: a copy warp (TMA boxes of one page each, and L2 prefetch of the next
// tile's pages, whose rows are contiguous), an MMA warp, two groups of four
// softmax warps that each take half of the rows (columns).  Shared memory: X
// (NR x 1152 B), a ring of 32 KB slots (128 positions x 128 channels) and the
// 16 KB slots of the shared key part, which hold P once the scores are done.
//
// What bounds it: a tile's 147 KB fill shared memory, so its chain is serial:
// P's product frees a slot, the next tile's rows arrive in it 1,100 to 2,400
// cycles later, scores, softmax (700 cycles).  A product step reads its
// 128-lane A operand and the columns' from shared memory (alone 32 cycles and a
// quarter of the columns, at 128 B a cycle; 68 steps a unit), and the copies
// write there meanwhile: 530 KB a unit at 48 columns, 4,200 cycles, and with
// the softmax between the products 5,200 to 5,600.  An SM's share of HBM brings
// a unit in 6,400: HBM bounds up to 64 rows.  Two CTAs side by side share the
// rows, which then come in 3,200: shared memory bounds 65 to 128 rows.
// Measured, a call with everything: 128 sequences of 8,000-8,192 tokens at 64
// heads 207 us (5.8 TB/s, 86 % of the measured copy); 131,072 and 100,001
// tokens at 32 heads 60 us (65 %); 64 sequences of 2,000-4,096 at 96 heads 74
// us (46 %); one of 1,000 at 16 heads 12 us (launches and one unit's chain).
#include <algorithm>

#include "latent_tc.cuh"

namespace kda {

using namespace tc;

// Error word of this file's kernels (bit 0: a bounded wait gave up, or
// cu_seqlens or a length broke its precondition; bit 1: a page index outside
// the cache).
__device__ unsigned int g_kda_latent_decode_error = 0;

namespace {

constexpr int kTile = 128;                // positions a unit
// Units that a row tile counts beside its tiles of positions, in front of them
// (queries, first scores, output).  24 sequences of 100-2,100 tokens with
// drafts: 26.0 us without, 24.3 with one, 24.5 with two; 64 of 2,000-4,096 at
// 96 heads: 75, 73, 74; 128 of 8,000-8,192 at 64 heads: 207, 208, 208.
constexpr int kExtra = 1;
constexpr int kMaxCtas = 160;             // grid bound (one CTA an SM; 152 SMs)
constexpr int kMaxSide = 8;               // row tiles of a token that CTAs take side by side
constexpr int kSoftWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + 2);
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr uint32_t kPair = 32768;         // 128 positions x 128 channels: [16 groups][2 blocks][8 rows][128 B]
constexpr uint32_t kRope = 16384;         // 128 positions x 64 channels; later P [128][64]
constexpr float kMoveAt = 8.f;            // log2 of the factor a score may pass the maximum by
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 0, TM_O = 64;   // S^T: 64 columns; O^T: 4 blocks of 64

// What a CTA leaves for the joining kernel: the row tile that starts in its
// units and goes on behind them.
struct Split {
    int32_t row;                          // first row (flat over [T * H])
    int32_t rows;                         // rows of the tile; 0: nothing
    int32_t pieces;                       // of it: here and in the CTAs `side` further on each
    int32_t blind;                        // its first rows, which see nothing
};

template <int NR>
struct Cfg {
    static constexpr int NP = NR == 64 || NR == 48 ? 4 : 5;   // 32 KB slots
    static constexpr int NQ = NR == 16 || NR == 48 ? 2 : 1;   // 16 KB slots
    static constexpr uint32_t X = 0;
    static constexpr uint32_t PAIR = NR * 1152u;
    static constexpr uint32_t ROPE = PAIR + NP * kPair;
    static constexpr uint32_t MISC = ROPE + NQ * kRope;
    static constexpr uint32_t BYTES = MISC + 4096;
    static_assert(BYTES + 1024 <= 232448, "shared memory of an SM");
};

// A sequence as the kernel sees it (clamped to what its buffers hold).
struct Seq {
    int row0, rows;                       // flat rows over [T * H], of this sequence
    int first;                            // positions its first new token sees (may be <= 0)
    int len, units, row_tiles;            // units: of each of its row tiles
};

struct Misc {
    uint64_t full_p[5], empty_p[5], full_r[2], empty_r[2];
    uint64_t x_full, x_empty, s_full, p_full, o_full, done;
    uint32_t tmem;
    int fail;
    uint32_t n_x, n_pair, n_rope;         // copies asked for, by barrier
    int b0, j0, t0;                       // first unit
    Seq seq0;                             // its sequence
    long long scan[kThreads / 32 + 1];
    long long start, units, each;         // this CTA's first unit and units; a group's units
    // per column (row of the tile), by softmax group
    float red[2][4][32];                  // cross-warp reductions
    alignas(16) float neg_m[2][32];       // minus the running maximum, log2 units
    alignas(16) float shift[2][32];       // how far the maximum moves
    alignas(16) float f[2][32];           // rescale factor, then 1 / sum
    alignas(16) int seen[2][32];                      // positions it may see
};
static_assert(sizeof(Misc) <= 4096, "control block");

struct Args {
    PagedRows pages;
    const int32_t *seq_lens, *cu;
    int N, T, H;
    int side;                             // CTAs side by side: row tiles of a token (one token a sequence)
    float scale_log2;                     // scale * log2 e
    __nv_bfloat16 *o;
    float *lse;
    Split *split;
    float *ws_lse;                        // [2 G][NR]
    float *ws_o;                          // [2 G][NR][512]
};

template <int NR>
__device__ __forceinline__ Seq get_seq(const Args &a, int b, bool flag) {
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
    if (bad && flag) atomicOr(&g_kda_latent_decode_error, kErrWait);
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
    __device__ __forceinline__ Walk(const Args &a, const Misc *m)
        : b(m->b0), j(m->j0), t(m->t0), left(m->units), u(m->start) {
        if (left > 0) s = m->seq0;
    }
    __device__ __forceinline__ bool next(const Args &a, Item &it) {
        int from, to;                     // tiles of positions
        do {
            if (left <= 0) return false;
            while (j >= s.row_tiles) {    // units are left, so a sequence with rows follows
                if (++b >= a.N) { left = 0; return false; }
                s = get_seq<NR>(a, b, false);
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

template <int NR>
__global__ void __launch_bounds__(kThreads, 1)
latent_decode_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_c,
                     const __grid_constant__ CUtensorMap map_r, const uint8_t *__restrict__ cache, const Args a) {
    using F = Cfg<NR>;
    constexpr int NC = NR / 2;                // columns of a softmax group
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Misc *M = reinterpret_cast<Misc *>(sm + F::MISC);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int cta = blockIdx.x, side = a.side;
    const int G = gridDim.x / side, group = cta / side;   // groups of CTAs side by side

    // ---- barriers and tensor memory, under the end of the kernel before this one
    if (t == 0) {
        M->fail = 0;
        M->b0 = M->j0 = M->t0 = 0;
        for (int i = 0; i < F::NP; ++i) { mbar_init(&M->full_p[i], 1); mbar_init(&M->empty_p[i], 1); }
        for (int i = 0; i < F::NQ; ++i) { mbar_init(&M->full_r[i], 1); mbar_init(&M->empty_r[i], 1); }
        mbar_init(&M->x_full, 1);
        mbar_init(&M->x_empty, 1);
        mbar_init(&M->s_full, 1);
        mbar_init(&M->p_full, kSoftWarps);
        mbar_init(&M->o_full, 1);
        mbar_init(&M->done, 1);
        fence_mbar_init();
    }
    if (warp == kSoftWarps) tmem_alloc(&M->tmem, kTmemCols);
    if (warp == kSoftWarps + 1 && lane == 0) {
        prefetch_tmap(&map_x);
        prefetch_tmap(&map_c);
        prefetch_tmap(&map_r);
    }
    wait_for_previous();
    // ---- this CTA's units: a block-wide scan of the sequences' units
    {
        const int per = (a.N + kThreads - 1) / kThreads;
        const int b_lo = min(a.N, t * per), b_hi = min(a.N, b_lo + per);
        long long mine = 0;
        Seq s;                                         // the only one where there are few
        for (int b = b_lo; b < b_hi; ++b) {
            s = get_seq<NR>(a, b, cta == 0);           // CTA 0 flags what is wrong with a sequence
            mine += (long long)s.units * s.row_tiles;
        }
        long long incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) M->scan[warp] = incl;
        if (t == 0) a.split[cta] = Split{0, 0, 0, 0};
        __syncthreads();
        long long before = incl - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += M->scan[w];
            total += M->scan[w];
        }
        // as many units for each group as the one with the most must have: fewer groups, and fewer
        // pieces, where that leaves some without
        const long long each = max(1LL, (total + G - 1) / G);
        const long long u0 = min(total, group * each), u1 = group < G ? min(total, u0 + each) : u0;
        if (t == 0) {
            M->units = u1 - u0;
            M->start = u0;
            M->each = each;
        }
        if (u1 > u0 && u0 >= before && u0 < before + mine) {
            for (int b = b_lo; b < b_hi; ++b) {
                if (per > 1) s = get_seq<NR>(a, b, false);
                const long long n = (long long)s.units * s.row_tiles;
                if (u0 < before + n) {
                    M->b0 = b;
                    M->seq0 = s;
                    M->j0 = (int)((u0 - before) / s.units);
                    M->t0 = (int)((u0 - before) % s.units);
                    break;
                }
                before += n;
            }
        }
    }
    let_next_begin();                         // the joining kernel
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;
    volatile int *fail = &M->fail;

    if (warp == kSoftWarps + 1) {
        // ================================================= copies
        Walk<NR> walk(a, M);
        Item it;
        uint32_t n_tile = 0, n_item = 0;          // tiles and items with tiles so far
        uint32_t n_x = 0, n_pair = 0, n_rope = 0; // copies asked for, by barrier
        const int page = 1 << a.pages.page_log2;
        const int brows = min(page, kTile), boxes = kTile / brows;   // TMA boxes down a tile
        bool ok = true;
        // the flat cache row of box `lane` of an item's tile `i` (P * page: past the end, reads zeros)
        auto box_row = [&](const Item &of, int i, bool flag) -> int {
            const int pos = (of.tile + i) * kTile + lane * brows;
            if (lane >= boxes || pos >= of.len) return -1;
            const int64_t r = a.pages.row(of.b, pos);
            if (r < 0 && flag) atomicOr(&g_kda_latent_decode_error, kErrSlot);
            return r < 0 ? (int)(a.pages.P << a.pages.page_log2) : (int)r;
        };
        // A second walk, a tile in front, that only brings the rows into L2 (a page's rows are
        // contiguous): shared memory holds little more than one tile, which is busy while it is
        // computed with.  128 sequences of 8,000-8,192 tokens at 64 heads: 247 us a call without
        // it, 211 us one tile in front, asked for behind the present tile's own copies, 238 us
        // two and 319 us three tiles in front (more than L2 keeps for all the SMs).
        Walk<NR> ahead(a, M);
        Item ia;
        int i_ahead = 0, n_ahead = 0;
        bool more = true;
        auto prefetch = [&](bool issue) {
            while (more && i_ahead == n_ahead) {
                more = ahead.next(a, ia);
                i_ahead = 0;
                n_ahead = more ? ia.n : 0;
            }
            if (!more) return;
            const int rows = box_row(ia, i_ahead++, false);
            if (issue && rows >= 0 && rows < (a.pages.P << a.pages.page_log2))
                for (int e = 0; e < brows; e += 16)
                    bulk_prefetch_l2(cache + ((size_t)rows + e) * 1152u, 16 * 1152u);
        };
        while (ok && walk.next(a, it)) {
            if (it.n == 0) continue;
            int rows = box_row(it, 0, true);
            if (n_item > 0) ok = warp_wait(&M->x_empty, (n_item - 1) & 1, fail);
            if (!ok) break;
            ++n_x;
            if (lane == 0) {
                mbar_arrive_expect_tx(&M->x_full, NR * 1152u);
                for (int k = 0; k < 9; ++k)
                    tma_load_2d(sm + F::X + k * NR * 128u, &map_x, &M->x_full, 64 * k, it.row);
            }
            for (int i = 0; ok && i < it.n; ++i, ++n_tile) {
                const int live = __popc(__ballot_sync(0xffffffffu, rows >= 0));
                const int next_rows = i + 1 < it.n ? box_row(it, i + 1, true) : -1;
                for (int j = 0; j < 4; ++j) {
                    const uint32_t u = 4 * n_tile + j, slot = u % F::NP, use = u / F::NP;
                    if (use > 0) ok = warp_wait(&M->empty_p[slot], (use - 1) & 1, fail);
                    if (!ok) break;
                    ++n_pair;
                    if (lane == 0) mbar_arrive_expect_tx(&M->full_p[slot], (uint32_t)live * brows * 256u);
                    __syncwarp();
                    uint8_t *dst = sm + F::PAIR + slot * kPair;
                    if (rows >= 0) tma_load_4d(dst + lane * brows * 256u, &map_c, &M->full_p[slot], 0, 0, 2 * j, rows >> 3);
                    __syncwarp();
                }
                if (!ok) break;
                const uint32_t slot = n_tile % F::NQ, use = n_tile / F::NQ;
                if (use > 0) ok = warp_wait(&M->empty_r[slot], (use - 1) & 1, fail);
                if (!ok) break;
                ++n_rope;
                if (lane == 0) mbar_arrive_expect_tx(&M->full_r[slot], (uint32_t)live * brows * 128u);
                __syncwarp();
                if (rows >= 0)
                    tma_load_4d(sm + F::ROPE + slot * kRope + lane * brows * 128u, &map_r, &M->full_r[slot], 0, 0, kLatent / 64,
                                rows >> 3);
                __syncwarp();
                rows = next_rows;
                if (n_tile == 0) prefetch(false);          // the first tile itself
                prefetch(true);
            }
            ++n_item;
        }
        if (lane == 0) {
            M->n_x = n_x;
            M->n_pair = n_pair;
            M->n_rope = n_rope;
        }
    } else if (warp == kSoftWarps) {
        // ================================================= matrix products
        // the whole warp walks and waits, one lane issues
        Walk<NR> walk(a, M);
        Item it;
        uint32_t n_tile = 0, n_item = 0;
        bool ok = true;
        constexpr uint32_t id_s = instr_desc(kFmtBF16, 128, NR, 0, 0);
        constexpr uint32_t id_o = instr_desc(kFmtBF16, 128, NR, 1, 1);
        const Operand x_op = operand(sm + F::X, 16, 1024), k_op = operand(sm + F::PAIR, 16, 2048);
        const Operand v_op = operand(sm + F::PAIR, 1024, 2048), r_op = operand(sm + F::ROPE, 16, 1024);
        const uint32_t full_p = smem_u32(M->full_p), empty_p = smem_u32(M->empty_p);
        const uint32_t full_r = smem_u32(M->full_r), empty_r = smem_u32(M->empty_r);
        const uint32_t s_full = smem_u32(&M->s_full), p_full = smem_u32(&M->p_full);
        uint32_t slot = 0, lap = 0;               // next pair slot, its phase
        while (ok && walk.next(a, it)) {
            if (it.n == 0) continue;
            ok &= wait_or_fail(&M->x_full, n_item & 1, fail);
            for (int i = 0; i < it.n; ++i, ++n_tile) {
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                // S^T: channels 0..511 from the pairs, 512..575 from the shared part
                uint32_t at[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    at[j] = slot;
                    ok &= wait_or_fail(full_p + 8 * slot, lap, fail);
                    if (++slot == F::NP) { slot = 0; lap ^= 1; }
                    tc_fence_after();
                    const Operand k = k_op + at[j] * kPair;
                    if (elect_one()) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const Operand ke = k + ((e >> 2) * 1024u + (e & 3) * 32u);
                            const Operand xe = x_op + ((2 * j + (e >> 2)) * NR * 128u + (e & 3) * 32u);
                            if (j == 0 && e == 0) mma_ss<false>(tmem + TM_S, ke, xe, id_s, false);
                            else mma_ss<true>(tmem + TM_S, ke, xe, id_s);
                        }
                    }
                    __syncwarp();
                }
                const uint32_t rslot = n_tile % F::NQ;
                const Operand rope = r_op + rslot * kRope;
                ok &= wait_or_fail(full_r + 8 * rslot, (n_tile / F::NQ) & 1, fail);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mma_ss<true>(tmem + TM_S, rope + e * 32u, x_op + (8 * NR * 128u + e * 32u), id_s);
                    commit(s_full);
                    if (i + 1 == it.n && ok) mma_commit(&M->x_empty);
                }
                __syncwarp();
                // O^T += c^T P^T, a slot released as soon as its block is done (P's rows are one
                // 128-byte atom wide, so the shared part's descriptor serves it, 16 rows a step)
                ok &= wait_or_fail(p_full, n_tile & 1, fail);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Operand v = v_op + at[j] * kPair;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (e == 0) mma_ss<false>(tmem + TM_O + 64 * j, v, rope, id_o, i > 0);
                            else mma_ss<true>(tmem + TM_O + 64 * j, v + e * 4096u, rope + e * 2048u, id_o);
                        }
                        if (ok) commit(empty_p + 8 * at[j]);
                    }
                    if (ok) commit(empty_r + 8 * rslot);
                    if (i + 1 == it.n) mma_commit(&M->o_full);
                }
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, ok);         // one verdict, so that the warp stays together
            ++n_item;
        }
        // nothing of this CTA's products is in flight when its TMEM goes
        end_products(&M->done, fail);
    } else {
        // ================================================= softmax, output
        const int g = warp >> 2, quarter = warp & 3;
        const int col0 = g * NC;                        // this group's columns
        const uint32_t lane_base = (uint32_t)quarter << 21;   // 32 lanes a quarter, lane field at bit 16
        const int bar = 1 + g;
        const int pos_in_tile = quarter * 32 + lane;
        Walk<NR> walk(a, M);
        Item it;
        uint32_t n_tile = 0, n_item = 0;
        bool ok = true;
        while (ok && walk.next(a, it)) {
            float2 l[NC / 2];
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) l[c] = make_float2(0.f, 0.f);
            // (the barriers of the last item's output came after its last readers)
            if (quarter == 0 && lane < NC) {
                const int r = it.row_in_seq + col0 + lane;   // several new tokens differ in what they see
                M->seen[g][lane] = min(it.len, it.first_tok + r / a.H);
                // columns behind the tile's rows hold another sequence's queries, or what no sequence
                // has: a maximum of infinity (their exponents are -inf or NaN, which fmaxf leaves out)
                // takes them out of the vote below
                M->neg_m[g][lane] = col0 + lane < it.rows ? 0.f : -CUDART_INF_F;
            }
            bar_sync(bar, 128);
            // from here on a tile needs masks: the first row's limit
            const int all_see = min(it.len, it.first_tok + it.row_in_seq / a.H);
            for (int i = 0; i < it.n; ++i, ++n_tile) {
                const int p0 = (it.tile + i) * kTile;
                ok = warp_wait(&M->s_full, n_tile & 1, fail);
                tc_fence_after();
                float s[NC];
                tmem_ldn<NC>(tmem + lane_base + TM_S + col0, s);
                tmem_wait_ld();
                if (p0 + kTile > it.len) {
                    // rows behind the end: whatever the cache holds there must not meet a zero weight
                    const int from = it.len - p0;
                    for (int e = t; e < (kTile - from) * 64; e += kSoftThreads) {
                        const int r = from + (e >> 6), blk = (e >> 3) & 7, ch = e & 7;
                        const uint32_t slot = (4 * n_tile + (blk >> 1)) % F::NP;
                        *reinterpret_cast<uint4 *>(sm + F::PAIR + slot * kPair + (r >> 3) * 2048u + (blk & 1) * 1024u +
                                                   (r & 7) * 128u + ch * 16u) = make_uint4(0, 0, 0, 0);
                    }
                }
                // s <- s scale log2 e - m
                const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
                for (int c = 0; c < NC; c += 4) {
                    const float4 nm = *reinterpret_cast<const float4 *>(&M->neg_m[g][c]);
                    const float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), sc2, make_float2(nm.x, nm.y));
                    const float2 y = __ffma2_rn(make_float2(s[c + 2], s[c + 3]), sc2, make_float2(nm.z, nm.w));
                    s[c] = x.x; s[c + 1] = x.y; s[c + 2] = y.x; s[c + 3] = y.y;
                }
                if (p0 + kTile > all_see) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (p0 + pos_in_tile >= M->seen[g][c]) s[c] = -CUDART_INF_F;
                }
                float top = s[0];
#pragma unroll
                for (int c = 1; c < NC; ++c) top = fmaxf(top, s[c]);
                if (bar_any(bar, 128, top > kMoveAt || i == 0 || !ok)) {
                    // a new maximum for every column of the group
                    const float mx = lanes_reduce<NC, true>(s, lane);
                    if (lane < NC) M->red[g][quarter][lane] = mx;
                    if (bar_any(bar, 128, !ok)) { ok = false; break; }
                    if (quarter == 0 && lane < NC) {
                        float up = fmaxf(fmaxf(M->red[g][0][lane], M->red[g][1][lane]),
                                         fmaxf(M->red[g][2][lane], M->red[g][3][lane]));
                        // the first tile sets the maximum, later ones only raise it.  A row that
                        // sees nothing in its piece's first tile sees nothing in the later ones
                        // either: any finite maximum serves it
                        up = i > 0 ? fmaxf(up, 0.f) : up == -CUDART_INF_F ? 0.f : up;
                        const float was = M->neg_m[g][lane], now = was - up;
                        up = was - now;                // what the rounded maximum really moves by
                        M->neg_m[g][lane] = now;
                        M->shift[g][lane] = up;
                        M->f[g][lane] = i > 0 ? ex2_approx(-up) : 1.f;
                    }
                    bar_sync(bar, 128);
#pragma unroll
                    for (int c = 0; c < NC; ++c) s[c] -= M->shift[g][c];
#pragma unroll
                    for (int c = 0; c < NC / 2; ++c) {
                        l[c].x *= M->f[g][2 * c];
                        l[c].y *= M->f[g][2 * c + 1];
                    }
                    if (i > 0) {                       // the products before this tile are done (s_full)
#pragma unroll 1
                        for (int j = 0; j < 4; ++j) {
#pragma unroll 1
                            for (int c0 = 0; c0 < NC; c0 += 8) {
                                const uint32_t at = tmem + lane_base + TM_O + 64 * j + col0 + c0;
                                float ov[8];
                                tmem_ldn<8>(at, ov);
                                tmem_wait_ld();
#pragma unroll
                                for (int c = 0; c < 8; ++c) ov[c] *= M->f[g][c0 + c];
                                tmem_stn<8>(at, ov);
                            }
                        }
                        tmem_wait_st();
                    }
                }
                uint8_t *pr = sm + F::ROPE + (n_tile % F::NQ) * kRope + pos_in_tile * 128u;
#pragma unroll
                for (int c = 0; c < NC; c += 8) {
                    float p[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = ex2_approx(s[c + e]);
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        l[(c + e) / 2] = __fadd2_rn(l[(c + e) / 2], make_float2(p[e], p[e + 1]));
                    *reinterpret_cast<uint4 *>(pr + ((((col0 + c) >> 3) ^ (pos_in_tile & 7)) << 4)) = pack_bf8(p);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                if (!left_out(n_tile)) warp_arrive(&M->p_full);
            }
            if (!ok) break;
            // ---- the row tile's (piece's) output
            const bool whole = it.head && it.tail;
            const int slot = 2 * cta + (it.head ? 1 : 0);      // a piece that starts here goes on behind
            if (it.n > 0) {
                ok = warp_wait(&M->o_full, n_item & 1, fail);
                if (bar_any(bar, 128, !ok)) { ok = false; break; }
                tc_fence_after();
                ++n_item;
            }
            float ls[NC];
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) { ls[2 * c] = l[c].x; ls[2 * c + 1] = l[c].y; }
            const float part = lanes_reduce<NC, false>(ls, lane);
            if (lane < NC) M->red[g][quarter][lane] = part;
            bar_sync(bar, 128);
            if (quarter == 0 && lane < NC) {
                const float sum = (M->red[g][0][lane] + M->red[g][1][lane]) + (M->red[g][2][lane] + M->red[g][3][lane]);
                // A row that sees nothing has o = 0; one that sees positions has 1 / sum, NaN included,
                // and 0 / 0 where each of its scores is -inf.  A piece may be without weight: the
                // joining kernel tells
                const bool none = whole ? M->seen[g][lane] <= 0 : sum == 0.f;
                const float lg = none ? -CUDART_INF_F : log2f(sum) - M->neg_m[g][lane];
                M->f[g][lane] = none ? 0.f : 1.f / sum;
                if (col0 + lane < it.rows) {
                    if (!whole) a.ws_lse[slot * NR + col0 + lane] = lg;
                    else if (a.lse) a.lse[it.row + col0 + lane] = lg * 0.6931471805599453f;
                }
            }
            bar_sync(bar, 128);
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                float ov[NC];
                if (it.n > 0) {
                    tmem_ldn<NC>(tmem + lane_base + TM_O + 64 * j + col0, ov);
                    tmem_wait_ld();
                }
                const int ch = 128 * j + pos_in_tile;
#pragma unroll
                for (int c = 0; c < NC; ++c) ov[c] = it.n > 0 ? ov[c] * M->f[g][c] : 0.f;
                if (!whole) {
                    float *dst = a.ws_o + ((size_t)slot * NR + col0) * kLatent + ch;
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (col0 + c < it.rows) dst[(size_t)c * kLatent] = ov[c];
                } else {
                    // pairs of channels: even lanes store column c, odd lanes column c + 1
                    __nv_bfloat16 *dst = a.o + ((size_t)it.row + col0) * kLatent + (ch & ~1);
                    const bool odd = lane & 1;
#pragma unroll
                    for (int c = 0; c < NC; c += 2) {
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? ov[c] : ov[c + 1], 1);
                        const uint32_t two = odd ? pack_bf2(got, ov[c + 1]) : pack_bf2(ov[c], got);
                        if (col0 + c + odd < it.rows)
                            *reinterpret_cast<uint32_t *>(dst + (size_t)(c + odd) * kLatent) = two;
                    }
                }
            }
            tc_fence_before();
            // the tile that starts here and goes on: who holds its last piece
            if (t == 0 && it.head && !it.tail) {
                const long long last = it.unit + it.tiles - 1;
                const int blind = min(it.rows, max(0, (1 - min(1, it.first_tok)) * a.H - it.row_in_seq));
                a.split[cta] = Split{it.row, it.rows, (int)(last / M->each) - group + 1, blind};
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*fail) {                          // a role gave up: nobody may have waited for the last copies
        if (t == 0) atomicOr(&g_kda_latent_decode_error, kErrWait);
        if (warp == kSoftWarps + 1) {
            land(&M->x_full, M->n_x, 1);
            land(M->full_p, M->n_pair, F::NP);
            land(M->full_r, M->n_rope, F::NQ);
        }
    }
    if (warp == kSoftWarps) tmem_dealloc(tmem, kTmemCols);
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

template <int NR>
cudaError_t launch(const CUtensorMap &mx, const CUtensorMap &mc, const CUtensorMap &mr, const void *cache, const Args &a,
                   cudaStream_t stream) {
    static KernelSetup setup;
    int sms = 0;
    cudaError_t e = setup.get(reinterpret_cast<const void *>(latent_decode_kernel<NR>), Cfg<NR>::BYTES + 1024, &sms);
    if (e != cudaSuccess) return e;
    const int G = std::min(sms, kMaxCtas);
    e = launch_early(latent_decode_kernel<NR>, G, kThreads, Cfg<NR>::BYTES + 1024, stream, mx, mc, mr,
                     static_cast<const uint8_t *>(cache), a);
    if (e != cudaSuccess) return e;
    // 4 G blocks: all of them fit the SMs at once
    return launch_early(latent_join_kernel, 4 * G, kJoinThreads, 0, stream,
                        JoinArgs{a.split, a.ws_lse, a.ws_o, a.o, a.lse, NR, G, a.side});
}

}  // namespace

// Workspace: the split records, the pieces' log2-sum-exp, the pieces.
size_t latent_decode_workspace_bytes(int N, int64_t T, int H) {
    return kSplitBytes + kLseBytes + (size_t)2 * kMaxCtas * rows_of_tile(N, T, H) * kLatent * sizeof(float);
}

cudaError_t launch_latent_decode(const void *q, const void *cache, const int32_t *table,
                                 const int32_t *seq_lens, const int32_t *cu, float scale, void *o,
                                 float *lse, int N, int64_t T, int H, int64_t P, int page,
                                 int max_pages, void *ws, cudaStream_t stream) {
    const int NR = rows_of_tile(N, T, H);
    CUtensorMap mx, mc, mr;
    const uint32_t groups = (uint32_t)std::min(page, kTile) / 8;
    if (!make_map_rows(&mx, q, kLatentRow, T * H, kLatentRow, (uint32_t)NR) ||
        !make_map_groups(&mc, cache, kLatentRow, P * page, 2, groups) ||
        !make_map_groups(&mr, cache, kLatentRow, P * page, 1, groups))
        return cudaErrorInvalidValue;
    uint8_t *w = static_cast<uint8_t *>(ws);
    Args a;
    a.pages = paged_rows(table, P, page, max_pages);
    a.seq_lens = seq_lens;
    a.cu = cu;
    a.N = N;
    a.T = (int)T;
    a.H = H;
    // One token a sequence and more heads than a tile's rows: the row tiles of a sequence are taken
    // by neighbouring CTAs at the same time, so that its cached rows come from HBM once.  With
    // offsets the host does not know the sequences' row tiles, and a CTA walks them one after the
    // other: 64 sequences of 2,000-4,096 tokens at 96 heads 75 us without offsets, 91 us with them,
    // at 128 heads 82 and 97.
    const int row_tiles = cu ? 1 : (H + NR - 1) / NR;
    a.side = row_tiles <= kMaxSide ? row_tiles : 1;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    a.split = reinterpret_cast<Split *>(w);
    a.ws_lse = reinterpret_cast<float *>(w + kSplitBytes);
    a.ws_o = reinterpret_cast<float *>(w + kSplitBytes + kLseBytes);
    switch (NR) {
        case 16: return launch<16>(mx, mc, mr, cache, a, stream);
        case 32: return launch<32>(mx, mc, mr, cache, a, stream);
        case 48: return launch<48>(mx, mc, mr, cache, a, stream);
        default: return launch<64>(mx, mc, mr, cache, a, stream);
    }
}

cudaError_t read_latent_decode_error(unsigned int *code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kda_latent_decode_error, sizeof(unsigned int));
    if (e != cudaSuccess || !reset) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kda_latent_decode_error, &zero, sizeof(unsigned int));
}

#ifdef KDA_DEBUG
cudaError_t latent_decode_leave_out(unsigned int tile) { return set_leave_out(tile); }
#endif

}  // namespace kda
