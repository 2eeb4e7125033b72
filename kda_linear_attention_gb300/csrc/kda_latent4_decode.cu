// Absorbed latent attention of one or a few new tokens a sequence over the
// 4-bit paged cache, on the tensor cores.
//
// The products are those of the bf16 cache's decode, positions and then latent
// channels on the 128 TMEM lanes and the (token, head) rows as up to 64 columns:
//   S^T [128 positions x rows]   = K [128 x 576] X^T           (36 K-steps)
//   O^T [512 x rows]            += c^T [512 x 128] P^T         (4 blocks of 128 channels, 8 K-steps)
// A code times its scale has 6 significant bits and lies in fp16's range, so
// the latent operands are fp16, exactly what the cache stands for (but for its
// unit 2^exponent, which goes into the factors of S and O).  The queries become
// fp16 with a power of two a row that brings the row's largest magnitude to
// 2^14: what fp16 then loses is below 2^-38 of that.  The shared channels stay
// bf16 on both sides.  P is fp16 too: the running maximum is held at 2^7 and may
// be passed by a factor 2^8 before O^T and the sums are rescaled, so P is below
// 2^16, and what lies under fp16's normal numbers is below 2^-21 of the row's
// largest weight.  Sums are fp32, of the unrounded probabilities.
//
// Work is dealt out and pieces are joined as in latent_walk.cuh says.  Roles: an
// MMA warp, two groups of four softmax warps that each take half of the rows,
// and eight producer warps.  A producer thread has one position and half of its
// channels: it reads them straight from the pages (a whole sector a load, the
// next tile's as soon as a register is free, so a tile's time hides HBM), turns
// codes into fp16 once and writes them twice: into the 32 KB slot that the
// second product reads MN-major, and, as the first product's operand A, into
// TMEM, whose reads cost no shared-memory bandwidth.  TMEM holds S (up to 64
// columns), O (4 blocks), the shared channels (32) and as many blocks of 128
// channels (64 columns each) as fit beside them; the others are read K-major
// from their slot.
#include "latent4.cuh"
#include "latent_walk.cuh"

namespace kda {

using namespace tc;

// Error word of this file's kernels (bit 0: a bounded wait gave up, or
// cu_seqlens or a length broke its precondition; bit 1: a page index outside
// the cache).
__device__ unsigned int g_kda_latent4_decode_error = 0;

namespace {

constexpr int kSoftWarps = 8, kFeedWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + kFeedWarps + 1);
constexpr uint32_t kSlot = 32768;         // 128 positions x 128 channels: [16 groups][2 blocks][8 rows][128 B]
constexpr uint32_t kProbs = 16384;        // P [128][64]
constexpr float kLift = 7.f;              // log2 of what a row's largest weight is held at
constexpr float kMoveAt = 15.f;           // ... of what a weight may reach
constexpr uint32_t kTmemCols = 512;

template <int NR>
struct Cfg {
    // TMEM columns, every part at a multiple of 32
    static constexpr uint32_t S = 0, O = 64, OB = NR <= 32 ? 32 : 64, R = O + 4 * OB, K = R + 32;
    static constexpr int KB = NR <= 32 ? 4 : 2;                  // blocks of K in TMEM
    static_assert(K + 64 * KB <= kTmemCols, "tensor memory");
    // shared memory
    static constexpr uint32_t X = 0;
    static constexpr uint32_t C = NR * 1152u;
    static constexpr uint32_t P = C + 4 * kSlot;
    static constexpr uint32_t MISC = P + kProbs;
    static constexpr uint32_t BYTES = MISC + 4096;
    static_assert(BYTES + 1024 <= 232448, "shared memory of an SM");
};

struct Misc {
    uint64_t full[4], empty[4];           // a slot and its block of K
    uint64_t x_full, x_empty, s_full, p_full, o_full, done;
    uint32_t tmem;
    int fail;
    Begin begin;                          // this CTA's units
    alignas(16) float factor[2][64];      // of a row's scores, log2 units; row tiles in turn
    // per column (row of the tile), by softmax group
    float red[2][4][32];                  // cross-warp reductions
    alignas(16) float neg_m[2][32];       // minus the running maximum, log2 units
    alignas(16) float shift[2][32];       // how far the maximum moves
    alignas(16) float f[2][32];           // rescale factor, then the unit / sum
    alignas(16) int seen[2][32];          // positions it may see
};
static_assert(sizeof(Misc) <= 4096, "control block");

struct Args : Batch {
    const __nv_bfloat16 *q;
    const uint8_t *cache;
    int exponent;
    float scale_log2;                     // scale * log2 e * 2^exponent
    __nv_bfloat16 *o;
    float *lse;
    Split *split;
    float *ws_lse;                        // [2 G][NR]
    float *ws_o;                          // [2 G][NR][512]
};

// A sector (32 bytes) of global memory.
struct Sector {
    uint32_t w[8];
};
__device__ __forceinline__ void load_sector(Sector &s, const uint8_t *p, bool there) {
    if (there) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]), "=r"(s.w[4]), "=r"(s.w[5]),
                       "=r"(s.w[6]), "=r"(s.w[7])
                     : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s.w[i] = 0u;
    }
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Biased exponent of the largest magnitude of eight bf16 (255: not finite).
__device__ __forceinline__ uint32_t top8(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    return m >> 7;
}
__device__ __forceinline__ uint4 to_half8(uint4 u, float f) {
    float x[8];
    unpack_bf8(u, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= f;
    return pack_h8(x);
}
__device__ __forceinline__ uint4 scaled8(uint4 u, float f, float g) {
    float x[8];
    unpack_bf8(u, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * f * g;
    return pack_bf8(x);
}

template <int NR>
__global__ void __launch_bounds__(kThreads, 1)
latent4_decode_kernel(const Args a) {
    using F = Cfg<NR>;
    constexpr int NC = NR / 2;                // columns of a softmax group
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Misc *M = reinterpret_cast<Misc *>(sm + F::MISC);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int cta = blockIdx.x, group = cta / a.side;   // groups of CTAs side by side

    // ---- barriers and tensor memory, under the end of the kernel before this one
    if (t == 0) {
        M->fail = 0;
        for (int i = 0; i < 4; ++i) { mbar_init(&M->full[i], kFeedWarps); mbar_init(&M->empty[i], 1); }
        mbar_init(&M->x_full, kFeedWarps);
        mbar_init(&M->x_empty, 1);
        mbar_init(&M->s_full, 1);
        mbar_init(&M->p_full, kSoftWarps);
        mbar_init(&M->o_full, 1);
        mbar_init(&M->done, 1);
        fence_mbar_init();
    }
    if (warp == kThreads / 32 - 1) tmem_alloc(&M->tmem, kTmemCols);
    wait_for_previous();
    if (t == 0) a.split[cta] = Split{0, 0, 0, 0};
    find_units<NR, kThreads>(a, &M->begin, &g_kda_latent4_decode_error);
    let_next_begin();                         // the joining kernel
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;
    volatile int *fail = &M->fail;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;   // a warp's 32 TMEM lanes, lane field at bit 16

    if (warp == kThreads / 32 - 1) {
        // ================================================= matrix products
        // the whole warp walks and waits, one lane issues
        Walk<NR> walk(a, M->begin);
        Item it;
        uint32_t n_tile = 0, n_item = 0;
        bool ok = true;
        constexpr uint32_t id_s = instr_desc(kFmtF16, 128, NR, 0, 0);
        constexpr uint32_t id_r = instr_desc(kFmtBF16, 128, NR, 0, 0);
        constexpr uint32_t id_o = instr_desc(kFmtF16, 128, NR, 1, 1);
        const Operand x_op = operand(sm + F::X, 16, 1024), k_op = operand(sm + F::C, 16, 2048);
        const Operand v_op = operand(sm + F::C, 1024, 2048), p_op = operand(sm + F::P, 16, 1024);
        const uint32_t full = smem_u32(M->full), empty = smem_u32(M->empty);
        const uint32_t s_full = smem_u32(&M->s_full), p_full = smem_u32(&M->p_full);
        while (ok && walk.next(a, it)) {
            if (it.n == 0) continue;
            ok &= wait_or_fail(&M->x_full, n_item & 1, fail);
            for (int i = 0; i < it.n; ++i, ++n_tile) {
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                // S^T: the shared channels, which come with the first block, then the latent ones
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ok &= wait_or_fail(full + 8 * j, n_tile & 1, fail);
                    tc_fence_after();
                    if (elect_one()) {
                        if (j == 0) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mma_ts(tmem + F::S, tmem + F::R + 8 * e, x_op + (8 * NR * 128u + e * 32u), id_r, e > 0);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const Operand xe = x_op + ((2 * j + (e >> 2)) * NR * 128u + (e & 3) * 32u);
                            if (j < F::KB)
                                mma_ts(tmem + F::S, tmem + F::K + 64 * j + 8 * e, xe, id_s, true);
                            else
                                mma_ss<true>(tmem + F::S, k_op + (j * kSlot + (e >> 2) * 1024u + (e & 3) * 32u), xe, id_s);
                        }
                    }
                    __syncwarp();
                }
                if (elect_one()) {
                    commit(s_full);
                    if (i + 1 == it.n && ok) mma_commit(&M->x_empty);
                }
                __syncwarp();
                // O^T += c^T P^T, a slot released as soon as its block is done (P's rows are one
                // 128-byte atom wide, 16 rows a step)
                ok &= wait_or_fail(p_full, n_tile & 1, fail);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Operand v = v_op + j * kSlot;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (e == 0) mma_ss<false>(tmem + F::O + F::OB * j, v, p_op, id_o, i > 0);
                            else mma_ss<true>(tmem + F::O + F::OB * j, v + e * 4096u, p_op + e * 2048u, id_o);
                        }
                        if (ok) commit(empty + 8 * j);
                    }
                    if (i + 1 == it.n) mma_commit(&M->o_full);
                }
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, ok);         // one verdict, so that the warp stays together
            ++n_item;
        }
        // nothing of this CTA's products is in flight when its TMEM goes
        end_products(&M->done, fail);
    } else if (warp >= kSoftWarps) {
        // ================================================= producers
        const int w = warp - kSoftWarps, half = w >> 2;           // which 64 channels of each block
        const int p = 32 * (w & 3) + lane;                        // position in the tile, TMEM lane
        // the tiles, one in front of what is being written: its registers are loaded as they get free
        Walk<NR> walk(a, M->begin);
        Item it;
        int i = 0;
        it.n = it.tile = it.len = 0;
        bool more = true;
        const uint8_t *row = nullptr;                             // this thread's row; nullptr: none
        auto advance = [&]() {
            ++i;
            while (more && i >= it.n) {
                more = walk.next(a, it);
                i = 0;
            }
            row = nullptr;
            const int pos = (it.tile + i) * kTile + p;
            if (more && pos < it.len) {
                const int64_t r = a.pages.row(it.b, pos);
                if (r >= 0) row = a.cache + (size_t)r * kLatent4Row;
                else atomicOr(&g_kda_latent4_decode_error, kErrSlot);
            }
        };
        Sector codes[4], pe[2], scales;
        auto load_codes = [&](int j) { load_sector(codes[j], row + 64 * j + 32 * half, row != nullptr); };
        auto load_rest = [&]() {
            load_sector(scales, row + k4Scales, row != nullptr);
            load_sector(pe[0], row + k4Pe + 64 * half, row != nullptr);
            load_sector(pe[1], row + k4Pe + 64 * half + 32, row != nullptr);
        };
        i = -1;
        advance();
        if (more) {
            load_rest();
#pragma unroll
            for (int j = 0; j < 4; ++j) load_codes(j);
        }
        uint32_t n_tile = 0, n_item = 0;
        bool ok = true;
        while (more && ok) {
            if (i == 0) {
                // ---- a new row tile's queries: a warp a row
                if (n_item > 0) ok = warp_wait(&M->x_empty, (n_item - 1) & 1, fail);
                if (!ok) break;
#pragma unroll 2
                for (int r = w; r < NR; r += kFeedWarps) {
                    uint4 u[3] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                    if (r < it.rows) {
                        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (size_t)(it.row + r) * kLatentRow);
                        u[0] = __ldg(src + lane);
                        u[1] = __ldg(src + 32 + lane);
                        if (lane < 8) u[2] = __ldg(src + 64 + lane);
                    }
                    int top = (int)max(top8(u[0]), top8(u[1]));
                    const int tp = (int)top8(u[2]);
                    if (tp > 0) top = max(top, tp == 255 ? 255 : tp - a.exponent);
                    top = __reduce_max_sync(0xffffffffu, top);
                    // 2^e brings the row's largest magnitude to [2^14, 2^15); tiny rows to less
                    const int e = 141 - max(20, min(255, top));
                    const float f = pow2(e);
                    const int er = e - a.exponent, er1 = er / 2;
                    uint8_t *dst = sm + F::X + r * 128u;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int c = 32 * k + lane;
                        *reinterpret_cast<uint4 *>(dst + (c >> 3) * NR * 128u + (((c & 7) ^ (r & 7)) << 4)) = to_half8(u[k], f);
                    }
                    if (lane < 8)
                        *reinterpret_cast<uint4 *>(dst + 8 * NR * 128u + ((lane ^ (r & 7)) << 4)) =
                            scaled8(u[2], pow2(er1), pow2(er - er1));
                    if (lane == 0) M->factor[n_item & 1][r] = a.scale_log2 * pow2(-e);
                }
                fence_proxy_async_smem();
                warp_arrive(&M->x_full);
                ++n_item;
            }
            uint32_t s4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s4[j] = half ? scales.w[2 * j + 1] : scales.w[2 * j];
            uint32_t r16[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) { r16[k] = pe[0].w[k]; r16[8 + k] = pe[1].w[k]; }
            advance();                                            // the row that is loaded from here on
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (n_tile > 0) ok = warp_wait(&M->empty[j], (n_tile - 1) & 1, fail);
                if (!ok) break;
                tc_fence_after();
                if (j == 0) {
                    tmem_st8u(tmem + lane_base + F::R + 16 * half, r16);
                    tmem_st8u(tmem + lane_base + F::R + 16 * half + 8, r16 + 8);
                    if (more) load_rest();
                }
                uint8_t *dst = sm + F::C + j * kSlot + (p >> 3) * 2048u + half * 1024u + (p & 7) * 128u;
                const __half2 s01 = scales2(s4[j] & 0xffffu), s23 = scales2(s4[j] >> 16);
#pragma unroll
                for (int g = 0; g < 4; ++g) {                     // 16 channels of one scale
                    const __half2 s = g == 0   ? __half2half2(__low2half(s01))
                                      : g == 1 ? __half2half2(__high2half(s01))
                                      : g == 2 ? __half2half2(__low2half(s23))
                                               : __half2half2(__high2half(s23));
                    uint32_t v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = h2_bits(__hmul2(codes2((codes[j].w[2 * g + (e >> 2)] >> (8 * (e & 3))) & 0xffu), s));
                    if (j < F::KB) tmem_st8u(tmem + lane_base + F::K + 64 * j + 32 * half + 8 * g, v);
                    *reinterpret_cast<uint4 *>(dst + (((2 * g) ^ (p & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<uint4 *>(dst + (((2 * g + 1) ^ (p & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
                }
                if (more) load_codes(j);
                tmem_wait_st();
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive(&M->full[j]);
            }
            ++n_tile;
        }
    } else {
        // ================================================= softmax, output
        const int g = warp >> 2, quarter = warp & 3;
        const int col0 = g * NC;                        // this group's columns
        const int bar = 1 + g;
        const int pos_in_tile = quarter * 32 + lane;
        Walk<NR> walk(a, M->begin);
        Item it;
        uint32_t n_tile = 0, n_item = 0;
        bool ok = true;
        const float unit = pow2(a.exponent);
        while (ok && walk.next(a, it)) {
            float2 l[NC / 2];
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) l[c] = make_float2(0.f, 0.f);
            // (the barriers of the last item's output came after its last readers)
            if (quarter == 0 && lane < NC) {
                const int r = it.row_in_seq + col0 + lane;   // several new tokens differ in what they see
                M->seen[g][lane] = min(it.len, it.first_tok + r / a.H);
                // columns behind the tile's rows: a maximum of infinity takes them out of the vote below
                M->neg_m[g][lane] = col0 + lane < it.rows ? 0.f : -CUDART_INF_F;
            }
            bar_sync(bar, 128);
            // from here on a tile needs masks: the first row's limit
            const int all_see = min(it.len, it.first_tok + it.row_in_seq / a.H);
            const float *factor = M->factor[n_item & 1] + col0;
            for (int i = 0; i < it.n; ++i, ++n_tile) {
                const int p0 = (it.tile + i) * kTile;
                ok = warp_wait(&M->s_full, n_tile & 1, fail);
                tc_fence_after();
                float s[NC];
                tmem_ldn<NC>(tmem + lane_base + F::S + col0, s);
                tmem_wait_ld();
                // s <- s scale log2 e - m, with each row's factor
#pragma unroll
                for (int c = 0; c < NC; c += 4) {
                    const float4 nm = *reinterpret_cast<const float4 *>(&M->neg_m[g][c]);
                    const float4 sc = *reinterpret_cast<const float4 *>(&factor[c]);
                    const float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), make_float2(sc.x, sc.y), make_float2(nm.x, nm.y));
                    const float2 y = __ffma2_rn(make_float2(s[c + 2], s[c + 3]), make_float2(sc.z, sc.w), make_float2(nm.z, nm.w));
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
                                         fmaxf(M->red[g][2][lane], M->red[g][3][lane])) - kLift;
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
                                const uint32_t at = tmem + lane_base + F::O + F::OB * j + col0 + c0;
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
                uint8_t *pr = sm + F::P + pos_in_tile * 128u;
#pragma unroll
                for (int c = 0; c < NC; c += 8) {
                    float p[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = ex2_approx(s[c + e]);
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        l[(c + e) / 2] = __fadd2_rn(l[(c + e) / 2], make_float2(p[e], p[e + 1]));
                    *reinterpret_cast<uint4 *>(pr + ((((col0 + c) >> 3) ^ (pos_in_tile & 7)) << 4)) = pack_h8(p);
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
                M->f[g][lane] = none ? 0.f : unit / sum;
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
                    tmem_ldn<NC>(tmem + lane_base + F::O + F::OB * j + col0, ov);
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
    if (*fail && t == 0) atomicOr(&g_kda_latent4_decode_error, kErrWait);   // a role gave up
    if (warp == kThreads / 32 - 1) tmem_dealloc(tmem, kTmemCols);
}

template <int NR>
cudaError_t launch(const Args &a, cudaStream_t stream) {
    static KernelSetup setup;
    int sms = 0;
    cudaError_t e = setup.get(reinterpret_cast<const void *>(latent4_decode_kernel<NR>), Cfg<NR>::BYTES + 1024, &sms);
    if (e != cudaSuccess) return e;
    const int G = std::min(sms, kMaxCtas);
    e = launch_early(latent4_decode_kernel<NR>, G, kThreads, Cfg<NR>::BYTES + 1024, stream, a);
    if (e != cudaSuccess) return e;
    // 4 G blocks: all of them fit the SMs at once
    return launch_early(latent_join_kernel, 4 * G, kJoinThreads, 0, stream,
                        JoinArgs{a.split, a.ws_lse, a.ws_o, a.o, a.lse, NR, G, a.side});
}

}  // namespace

size_t latent4_decode_workspace_bytes(int N, int64_t T, int H) { return pieces_bytes(rows_of_tile(N, T, H)); }

cudaError_t launch_latent4_decode(const void *q, const void *cache, const int32_t *table,
                                  const int32_t *seq_lens, const int32_t *cu, float scale, int exponent,
                                  void *o, float *lse, int N, int64_t T, int H, int64_t P, int page,
                                  int max_pages, void *ws, cudaStream_t stream) {
    const int NR = rows_of_tile(N, T, H);
    uint8_t *w = static_cast<uint8_t *>(ws);
    Args a;
    a.pages = paged_rows(table, P, page, max_pages);
    a.seq_lens = seq_lens;
    a.cu = cu;
    a.N = N;
    a.T = (int)T;
    a.H = H;
    a.side = tiles_side_by_side(cu, H, NR);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.cache = static_cast<const uint8_t *>(cache);
    a.exponent = exponent;
    a.scale_log2 = scale * 1.4426950408889634f * pow2(exponent);
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    a.split = reinterpret_cast<Split *>(w);
    a.ws_lse = reinterpret_cast<float *>(w + kSplitBytes);
    a.ws_o = reinterpret_cast<float *>(w + kSplitBytes + kLseBytes);
    switch (NR) {
        case 16: return launch<16>(a, stream);
        case 32: return launch<32>(a, stream);
        case 48: return launch<48>(a, stream);
        default: return launch<64>(a, stream);
    }
}

cudaError_t read_latent4_decode_error(unsigned int *code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kda_latent4_decode_error, sizeof(unsigned int));
    if (e != cudaSuccess || !reset) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kda_latent4_decode_error, &zero, sizeof(unsigned int));
}

#ifdef KDA_DEBUG
cudaError_t latent4_decode_leave_out(unsigned int tile) { return set_leave_out(tile); }
#endif

}  // namespace kda
