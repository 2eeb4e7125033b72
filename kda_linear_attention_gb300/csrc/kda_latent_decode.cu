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
#include "latent_walk.cuh"

namespace kda {

using namespace tc;

// Error word of this file's kernels (bit 0: a bounded wait gave up, or
// cu_seqlens or a length broke its precondition; bit 1: a page index outside
// the cache).
__device__ unsigned int g_kda_latent_decode_error = 0;

namespace {

constexpr int kSoftWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + 2);
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr uint32_t kPair = 32768;         // 128 positions x 128 channels: [16 groups][2 blocks][8 rows][128 B]
constexpr uint32_t kRope = 16384;         // 128 positions x 64 channels; later P [128][64]
constexpr float kMoveAt = 8.f;            // log2 of the factor a score may pass the maximum by
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 0, TM_O = 64;   // S^T: 64 columns; O^T: 4 blocks of 64

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

struct Misc {
    uint64_t full_p[5], empty_p[5], full_r[2], empty_r[2];
    uint64_t x_full, x_empty, s_full, p_full, o_full, done;
    uint32_t tmem;
    int fail;
    uint32_t n_x, n_pair, n_rope;         // copies asked for, by barrier
    Begin begin;                          // this CTA's units
    // per column (row of the tile), by softmax group
    float red[2][4][32];                  // cross-warp reductions
    alignas(16) float neg_m[2][32];       // minus the running maximum, log2 units
    alignas(16) float shift[2][32];       // how far the maximum moves
    alignas(16) float f[2][32];           // rescale factor, then 1 / sum
    alignas(16) int seen[2][32];                      // positions it may see
};
static_assert(sizeof(Misc) <= 4096, "control block");

struct Args : Batch {
    float scale_log2;                     // scale * log2 e
    __nv_bfloat16 *o;
    float *lse;
    Split *split;
    float *ws_lse;                        // [2 G][NR]
    float *ws_o;                          // [2 G][NR][512]
};

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
    const int group = cta / side;             // groups of CTAs side by side

    // ---- barriers and tensor memory, under the end of the kernel before this one
    if (t == 0) {
        M->fail = 0;
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
    if (t == 0) a.split[cta] = Split{0, 0, 0, 0};
    find_units<NR, kThreads>(a, &M->begin, &g_kda_latent_decode_error);
    let_next_begin();                         // the joining kernel
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;
    volatile int *fail = &M->fail;

    if (warp == kSoftWarps + 1) {
        // ================================================= copies
        Walk<NR> walk(a, M->begin);
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
        Walk<NR> ahead(a, M->begin);
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
        Walk<NR> walk(a, M->begin);
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
        Walk<NR> walk(a, M->begin);
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
                a.split[cta] = Split{it.row, it.rows, (int)(last / M->begin.each) - group + 1, blind};
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
size_t latent_decode_workspace_bytes(int N, int64_t T, int H) { return pieces_bytes(rows_of_tile(N, T, H)); }

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
    a.side = tiles_side_by_side(cu, H, NR);
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
