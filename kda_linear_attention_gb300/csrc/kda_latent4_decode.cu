// Absorbed latent attention of one or a few new tokens a sequence over the
// 4-bit paged cache, on the tensor cores.
//
// The products are those of the bf16 cache's decode, positions and then latent
// channels on the 128 TMEM lanes and the (token, head) rows as up to 64 columns:
//   S^T [128 positions x rows]   = K [128 x 576] X^T           (36 K-steps)
//   O^T [512 x rows]            += c^T [512 x 128] P^T         (4 blocks of 128 channels, 8 K-steps)
// A code times its scale has 6 significant bits and lies in fp16's range, so
// the latent operands are fp16, exactly what the cache stands for (but for its
// unit 2^exponent, which goes into the factors of S and O).  The queries' latent
// channels become fp16 with a power of two a row that brings the row's largest
// magnitude to 2^14: what fp16 then loses is below 2^-38 of that.  The shared
// channels stay bf16 on both sides, the queries' with 2^-exponent on top of that
// power, so that their products are in the latent ones' unit.  At an exponent above
// 0 they count among the row's magnitudes with it; below 0 without it, and then
// reach 2^47, for which bf16 and fp32 have room (counted with it they took the row's
// range: scores of rows whose two parts count alike were off by 0.01 at -32).
// P is fp16 too: the running maximum is held at 2^7 and may be passed by a factor
// 2^8 before O^T and the sums are rescaled, so P is below 2^16, and what lies under
// fp16's normal numbers is below 2^-21 of the row's largest weight.  Sums are fp32,
// of the unrounded probabilities.
//
// Work is dealt out and pieces are joined as latent_walk.cuh says.  Sixteen
// warps, which leaves a thread 128 registers:
//   - two groups of four softmax warps that each take half of the rows.  The
//     first of them issues the products: between a tile's P and the next tile's
//     scores it has nothing else to do;
//   - two groups of four producer warps, one for the even blocks of 128 channels
//     and one for the odd ones.  Four lanes take a position's 64 bytes of codes of
//     a block, turn them into fp16 and write them into the block's 32 KB slot,
//     which is both products' operand A, K-major for the first, MN-major for the
//     second.
// A slot is free as soon as its block of the second product is done, and a
// block's scores begin as soon as it is written; a block is turned into fp16
// before its slot is free.
//
// A producer thread copies what it will read next into 64 bytes of its own
// (cp.async, which needs no register and no line of the first-level cache:
// beside 227 KB of shared memory that holds some 200), and reads it when its
// block's turn comes; the rows are on their way from HBM to L2 a tile before.
// Beside 64 rows' queries there is no room for that, and the next 64 bytes are
// loaded into registers (64 sequences of 2,000-4,096 tokens at 96 heads, tiles of
// 48 rows: 111 us so, 95 through shared memory; 128 of 8,000-8,192 at 64 heads:
// two tiles of 32 rows through shared memory 356 us, one of 64 261 us).
// The shared-memory writes of all roles are ordered before the tensor core's
// reads by the warp that issues the products, between having seen the arrivals
// and issuing: a fence in the writing threads waits for their copies in flight
// (the same time within 1 %, and 400 to 600 cycles longer a softmax).
//
// What bounds it: a tile's chain.  By one block's clock, from scores to scores,
// 5,600 cycles at 16 rows, 6,200 at 32, 6,800 at 48 and 8,400 at 64: softmax up to
// its arrival (840 at 16 rows, 1,750 at 64), the second product up to the slot that
// frees first (920, 1,270), its block's stores (1,030, 1,400), the other blocks'
// conversion and stores (1,880, 2,700), the last scores (920, 1,330).  Of these
// 2,200 are the products' reads of their operands from shared memory, at 128 B a
// cycle, 1,000 the converted codes' writes and 500 a scheduler the conversions, 9
// instructions a word.  The producers' own instructions, some 1,000 a tile and warp
// at one in five cycles, are as long as the chain.  Over whole calls (152 sequences
// of 512 to 8,192 tokens, in a graph) a tile comes to 3.0, 3.2, 3.5 and 4.5 us, and
// 13, 18, 21 and 22 us are beside the tiles: launches, page lookups, first rows and
// queries, pieces out and joined.  Measured and not kept: codes turned into fp16 by shifts and masks
// (19 instructions a word); the roles' loops unrolled (twice the time: the
// instruction cache); rows brought by TMA in boxes of 64 bytes (900 rows' requests
// a tile: 2,000 cycles from asking to arrival); all warps taking turns at the
// softmax and the next tile (440 us where this takes 260: what comes next as
// loads in 16 warps); sixteen producer warps (60 us where this takes 56); K as
// the first product's operand in TMEM, which saves 1,000 cycles of shared-memory
// reads a tile (92 us where this takes 95, 55 where 56).
// Measured, a call with everything: 128 sequences of 8,000-8,192 tokens at 64
// heads 261 us (the bf16 cache: 208); 64 of 2,000-4,096 at 96 heads 95 us (74);
// 131,072 and 100,001 at 32 heads 56 us (60); 24 of 100-2,100 with drafts 27 us
// (23); one of 1,000 at 16 heads 14 us (13).
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
constexpr int kThreads = 32 * (kSoftWarps + kFeedWarps);
constexpr uint32_t kSlot = 32768;         // 128 positions x 128 channels: [16 groups][2 blocks][8 rows][128 B]
constexpr uint32_t kProbs = 16384;        // P [128][64], the shared channels [128][64]
constexpr float kLift = 7.f;              // log2 of what a row's largest weight is held at
constexpr float kMoveAt = 15.f;           // ... of what a weight may reach
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kMisc = 4096;

constexpr uint32_t TM_S = 0, TM_O = 64;   // S^T: 64 columns; O^T: 4 blocks of 64

constexpr uint32_t kAhead = 64 * 32 * kFeedWarps;   // 64 bytes a producer thread
constexpr uint32_t kScales = 1024 * kFeedWarps;     // of 32 rows, a warp

template <int NR>
struct Cfg {
    static constexpr uint32_t X = 0;
    static constexpr uint32_t C = NR * 1152u;
    static constexpr uint32_t P = C + 4 * kSlot;                 // the shared channels, then P
    // what is copied ahead has a place in shared memory where the queries leave one, else registers
    static constexpr bool STAGED = NR <= 48;
    static constexpr uint32_t RAW = P + kProbs;
    static constexpr uint32_t SC = RAW + (STAGED ? kAhead : 0);
    static constexpr uint32_t MISC = SC + (STAGED ? kScales : 0);
    static constexpr uint32_t STEPS = MISC + kMisc;   // the softmax warps' walks, where registers are short
    static constexpr uint32_t BYTES = STEPS + (STAGED ? 0 : kSoftWarps * 128u);
    static_assert(BYTES + 1024 <= 232448, "shared memory of an SM");
};

// A warp's walk over the row tiles, which lies in shared memory: it is looked at
// once a row tile, and a thread's registers are for what a tile needs.  Lane 0
// walks.
struct Steps {
    alignas(16) unsigned char walk[64];   // a Walk<NR>
    Item it;
};
template <int NR>
__device__ __forceinline__ void begin_steps(Steps *s, const Batch &a, const Begin &b) {
    static_assert(sizeof(Walk<NR>) <= sizeof(s->walk), "room for a walk");
    if ((threadIdx.x & 31) == 0) *reinterpret_cast<Walk<NR> *>(s->walk) = Walk<NR>(a, b);
    __syncwarp();
}
template <int NR>
__device__ __forceinline__ bool next_step(Steps *s, const Batch &a) {
    int more = 0;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        Walk<NR> w = *reinterpret_cast<Walk<NR> *>(s->walk);
        Item it;
        more = w.next(a, it);
        *reinterpret_cast<Walk<NR> *>(s->walk) = w;
        if (more) s->it = it;
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, more, 0) != 0;
}

struct Misc {
    uint64_t full[4], empty[4];           // a slot
    uint64_t s_full, p_full, o_full, x_full, done;   // (up to o_full in this order: Products)
    uint32_t tmem;
    int fail;
    Begin begin;                          // this CTA's units
    Steps steps[kFeedWarps];              // by producer warp
    alignas(16) float factor[2][64];      // of a row's scores, log2 units; row tiles in turn
    // per column (row of the tile), by softmax group
    float red[2][4][32];                  // cross-warp reductions
    alignas(16) float neg_m[2][32];       // minus the running maximum, log2 units
    alignas(16) float shift[2][32];       // how far the maximum moves
    alignas(16) float f[2][32];           // rescale factor, then the unit / sum
    alignas(16) int seen[2][32];          // positions it may see
};
static_assert(sizeof(Misc) <= kMisc, "control block");

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

// 16 bytes global -> shared past the first-level cache; zeros where `there` is not.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void load16(uint4 &v, const uint8_t *p, bool there) {
    v = make_uint4(0u, 0u, 0u, 0u);
    if (there)
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
}
__device__ __forceinline__ void load2(uint32_t &v, const uint8_t *p, bool there) {
    uint16_t two = 0;
    if (there) asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(two) : "l"(p));
    v = two;
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
// The codes of a word times their scale.  The conversions take a word's bytes as
// they are: with the multiplications a word costs 9 instructions (shifts and masks
// that build fp16 numbers: 19).
__device__ __forceinline__ uint4 halves8(uint32_t w, __half2 s) {
    uint32_t a, b, c, d;
    asm("{\n\t.reg .b8 p, q, r, t;\n\t"
        "mov.b32 {p, q, r, t}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, p;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, r;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, t;\n\t}"
        : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
        : "r"(w));
    return make_uint4(h2_bits(__hmul2(h2_of(a), s)), h2_bits(__hmul2(h2_of(b), s)), h2_bits(__hmul2(h2_of(c), s)),
                      h2_bits(__hmul2(h2_of(d), s)));
}
__device__ __forceinline__ uint4 scaled8(uint4 u, float f, float g) {
    float x[8];
    unpack_bf8(u, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * f * g;
    return pack_bf8(x);
}

// The products of a tile, issued by one lane of a warp that stays together.  The
// operands are laid down once: a product is issued every 40 cycles or so.
template <int NR>
struct Products {
    using F = Cfg<NR>;
    Operand x, k, v, p;
    uint32_t tmem, bars;                  // bars: full, empty, s_full, p_full, o_full
    volatile int *fail;

    __device__ __forceinline__ Products(uint8_t *sm, Misc *M, uint32_t tm)
        : x(operand(sm + F::X, 16, 1024)), k(operand(sm + F::C, 16, 2048)), v(operand(sm + F::C, 1024, 2048)),
          p(operand(sm + F::P, 16, 1024)), tmem(tm), bars(smem_u32(M->full)), fail(&M->fail) {}
    static constexpr uint32_t kFull = 0, kEmpty = 32, kS = 64, kP = 72, kO = 80;

    __device__ __forceinline__ bool seen(uint32_t bar, uint32_t n) const { return wait_or_fail(bars + bar, n & 1, fail); }
    __device__ __forceinline__ void ordered() const {
        fence_proxy_async_smem();
        tc_fence_after();
    }
    // S^T of tile n, block by block as they are written; the shared channels come with the last two.
    __device__ __forceinline__ bool scores(uint32_t n) const {
        constexpr uint32_t id = instr_desc(kFmtF16, 128, NR, 0, 0), id_r = instr_desc(kFmtBF16, 128, NR, 0, 0);
        bool ok = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ok &= seen(kFull + 8 * j, n);
            ordered();
            if (elect_one()) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const Operand ke = k + (j * kSlot + (e >> 2) * 1024u + (e & 3) * 32u);
                    const Operand xe = x + ((2 * j + (e >> 2)) * NR * 128u + (e & 3) * 32u);
                    if (j == 0 && e == 0) mma_ss<false>(tmem + TM_S, ke, xe, id, false);
                    else mma_ss<true>(tmem + TM_S, ke, xe, id);
                }
                if (j == 3) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) mma_ss<true>(tmem + TM_S, p + e * 32u, x + (8 * NR * 128u + e * 32u), id_r);
                    commit(bars + kS);
                }
            }
            __syncwarp();
        }
        return __all_sync(0xffffffffu, ok);
    }
    // O^T += c^T P^T, a slot released as soon as its block is done (P's rows are one 128-byte atom
    // wide, 16 rows a step).
    __device__ __forceinline__ bool output(uint32_t n, bool acc, bool last) const {
        constexpr uint32_t id = instr_desc(kFmtF16, 128, NR, 1, 1);
        const bool ok = __all_sync(0xffffffffu, seen(kP, n));
        ordered();
        if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Operand vj = v + j * kSlot;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (e == 0) mma_ss<false>(tmem + TM_O + 64 * j, vj, p, id, acc);
                    else mma_ss<true>(tmem + TM_O + 64 * j, vj + e * 4096u, p + e * 2048u, id);
                }
                if (ok) commit(bars + kEmpty + 8 * j);
            }
            if (last) commit(bars + kO);
        }
        __syncwarp();
        return ok;
    }
};

template <int NR>
__global__ void __launch_bounds__(kThreads, 1)
latent4_decode_kernel(const __grid_constant__ Args a) {
    using F = Cfg<NR>;
    constexpr int NC = NR / 2;                // columns of a softmax group
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Misc *M = reinterpret_cast<Misc *>(sm + F::MISC);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int cta = blockIdx.x;

    // ---- barriers and tensor memory, under the end of the kernel before this one
    if (t == 0) {
        M->fail = 0;
        for (int i = 0; i < 4; ++i) { mbar_init(&M->full[i], kFeedWarps / 2); mbar_init(&M->empty[i], 1); }
        mbar_init(&M->x_full, kFeedWarps);
        mbar_init(&M->s_full, 1);
        mbar_init(&M->p_full, kSoftWarps);
        mbar_init(&M->o_full, 1);
        mbar_init(&M->done, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&M->tmem, kTmemCols);
    wait_for_previous();
    if (t == 0) a.split[cta] = Split{0, 0, 0, 0};
    find_units<NR, kThreads>(a, &M->begin, &g_kda_latent4_decode_error);
    let_next_begin();                         // the joining kernel
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;
    volatile int *fail = &M->fail;

    if (warp >= kSoftWarps) {
        // ================================================= producers
        const int w = warp - kSoftWarps;
        // Four warps a block, the first four the even ones: rows 32 (w % 4) + 8 k + pr of a tile, 32 of the
        // block's channels
        const int half = w >> 2, row0 = 32 * (w & 3) + (lane >> 2), pr = lane >> 2, pc = lane & 3;
        bool ok = true;
        uint32_t n_tile = 0, n_item = 0;
        // ---- the tiles: tile `at` of row tile `it` is the next one, whose rows are copied ahead
        Steps *const steps = &M->steps[w];
        begin_steps<NR>(steps, a, M->begin);
        const Item &it = steps->it;
        int at = -1, tiles = 0;
        bool more = true;
        // pages of a lane's row 32 (w % 4) + lane of it, and of that of the tile behind it in the row tile
        // (-1: none); asked for by look(), waited for in turn_to()
        int page_of = 0, page_ahead = 0, rows[4];       // rows: this thread's rows in the cache, -1: none
        bool there = false, there_ahead = false;
        auto place = [&]() { return (it.tile + at) * kTile + 32 * (w & 3) + lane; };
        auto look = [&]() {
            ++at;
            while (more && at >= tiles) {
                more = next_step<NR>(steps, a);
                tiles = more ? it.n : 0;
                at = 0;
            }
            if (!more) return;
            const int pos = place();
            const int32_t *const table = a.pages.table + (size_t)it.b * a.pages.max_pages;
            there = pos < it.len;
            there_ahead = half == 0 && (lane & 15) == 0 && at + 1 < tiles && pos + kTile < it.len;
            if (there) page_of = table[pos >> a.pages.page_log2];
            if (there_ahead) page_ahead = table[(pos + kTile) >> a.pages.page_log2];
        };
        auto turn_to = [&]() {
            const int in_page = place() & ((1 << a.pages.page_log2) - 1);
            const bool good = there && page_of >= 0 && page_of < a.pages.P;
            if (there && !good && half == 0) atomicOr(&g_kda_latent4_decode_error, kErrSlot);
            const int mine = good ? (page_of << a.pages.page_log2) + in_page : -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) rows[k] = __shfl_sync(0xffffffffu, mine, 8 * k + pr);
            // its rows on their way to L2: a page holds 16 in a row at least
            if (there_ahead && page_ahead >= 0 && page_ahead < a.pages.P) {
                const size_t r = ((size_t)page_ahead << a.pages.page_log2) + ((place() + kTile) & ((1 << a.pages.page_log2) - 1));
                bulk_prefetch_l2(a.cache + r * kLatent4Row, 16 * kLatent4Row);
            }
        };
        // what comes next, 16 bytes of each of this thread's rows (codes of a block, then shared channels),
        // and the scales
        uint4 next[4];
        uint32_t scales[4];
        const uint32_t ahead = smem_u32(sm + F::RAW) + (t - 32 * kSoftWarps) * 16u;
        const uint32_t scales_at = smem_u32(sm + F::SC) + w * 1024u;
        auto row = [&](int k) { return a.cache + (size_t)(rows[k] < 0 ? 0 : rows[k]) * kLatent4Row; };
        auto copy = [&](int from) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (F::STAGED) copy16(ahead + k * (kAhead / 4), row(k) + from + 16 * pc, rows[k] >= 0);
                else load16(next[k], row(k) + from + 16 * pc, rows[k] >= 0);
            }
        };
        auto copy_scales = [&](int j) {                 // of block j; staged ones of all blocks with the first
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (F::STAGED) {
                    if (pc < 2 && j < 2) copy16(scales_at + (8 * k + pr) * 32u + 16 * pc, row(k) + k4Scales + 16 * pc, rows[k] >= 0);
                } else {
                    load2(scales[k], row(k) + k4Scales + 8 * j + 2 * pc, rows[k] >= 0);
                }
            }
        };
        auto take = [&]() {
            if constexpr (F::STAGED) {
                copies_done();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(next[k].x), "=r"(next[k].y), "=r"(next[k].z), "=r"(next[k].w)
                                 : "r"(ahead + k * (kAhead / 4)));
            }
        };
        auto take_scales = [&](int j) {
            if constexpr (F::STAGED) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    scales[k] = *reinterpret_cast<const uint16_t *>(sm + F::SC + w * 1024u + (8 * k + pr) * 32u + 8 * j + 2 * pc);
            }
        };
        // The upper 64 channels' lanes take their words in another order, so that eight lanes that write
        // together meet in no bank.
        const bool turn = pc & 2;
        uint8_t *const my_slot = sm + F::C + (row0 >> 3) * 2048u + (pc >> 1) * 1024u + pr * 128u;
        uint8_t *const my_shared = sm + F::P + row0 * 128u;
        look();
        bool now = more, fresh = more;                  // there is a tile at hand; it is its row tile's first
        if (more) {
            turn_to();
            copy(64 * half);
            copy_scales(half);
        }
        while (now && ok) {
            if (fresh) {
                // ---- a new row tile's queries, a warp a row; the last one's scores are done
                if (n_tile > 0) ok = warp_wait(&M->s_full, (n_tile - 1) & 1, fail);
                if (!ok) break;
#pragma unroll 1
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
                    if (tp > 0) top = max(top, tp == 255 ? 255 : tp - max(a.exponent, 0));
                    top = __reduce_max_sync(0xffffffffu, top);
                    // 2^e brings the row's largest magnitude to [2^14, 2^15); tiny rows to less.  The shared
                    // part at 2^er stays below 2^(15 - min(0, exponent))
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
                warp_arrive(&M->x_full);
                ++n_item;
            }
            take();
            if (F::STAGED) copy(64 * half + 128);       // what comes next: this warp's other block
            look();
            // ---- its blocks, each in fp16 before its slot is free.  One copy of this code and not four:
            // unrolled, the roles' code does not fit the instruction cache, which takes twice the time
#pragma unroll 1
            for (int j = half; j < 4; j += 2) {
                uint4 v[4][4];
                take_scales(j);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 c = next[k];
                    const __half2 s = scales2(scales[k]);
                    const __half2 s0 = turn ? __high2half2(s) : __low2half2(s), s1 = turn ? __low2half2(s) : __high2half2(s);
                    v[k][0] = halves8(turn ? c.z : c.x, s0);
                    v[k][1] = halves8(turn ? c.w : c.y, s0);
                    v[k][2] = halves8(turn ? c.x : c.z, s1);
                    v[k][3] = halves8(turn ? c.y : c.w, s1);
                }
                if constexpr (F::STAGED) {
                    take();                             // the other block, then a half of the shared channels
                    if (j < 2) copy(k4Pe + 64 * half);
                } else {
                    copy(j < 2 ? 64 * j + 128 : k4Pe + 64 * half);
                    if (j < 2) copy_scales(j + 2);
                }
                if (n_tile > 0) ok &= warp_wait(&M->empty[j < 2 ? j : 3], (n_tile - 1) & 1, fail);   // with 3, P's place
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4 *>(my_slot + j * kSlot + k * 2048u +
                                                   (((4 * (pc & 1) + (e ^ (turn ? 2 : 0))) ^ pr) << 4)) = v[k][e];
                if (j >= 2) {                           // a half of the shared channels, where P was
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4 *>(my_shared + k * 1024u + (((4 * half + pc) ^ pr) << 4)) = next[k];
                }
                warp_arrive(&M->full[j]);
            }
            fresh = at == 0;                            // the next tile
            now = more;
            if (more) {
                __syncwarp();                           // the warp's scales have been read
                turn_to();
                copy(64 * half);
                copy_scales(half);
            }
            ++n_tile;
        }
        copies_done();                                  // none is in flight when the block ends
    } else {
        // ================================================= softmax, output; warp 0 issues the products
        const Products<NR> mma(sm, M, tmem);
        const int g = warp >> 2, quarter = warp & 3;
        const int col0 = g * NC;                        // this group's columns
        const int bar = 1 + g;
        const int p = quarter * 32 + lane;              // position in a tile, TMEM lane
        const uint32_t lanes = tmem + ((uint32_t)quarter << 21);   // 32 lanes a quarter, lane field at bit 16
        uint32_t n_tile = 0, n_item = 0;
        bool ok = true;
        bool lost = false;                              // the group's verdict: a warp's own `ok` ends nothing alone
        Steps *const steps = reinterpret_cast<Steps *>(sm + F::STEPS) + warp;
        if constexpr (!F::STAGED) begin_steps<NR>(steps, a, M->begin);
        Walk<NR> walk(a, M->begin);
        Item own;
        const Item &it = F::STAGED ? own : steps->it;
        auto next = [&]() {
            if constexpr (F::STAGED) return walk.next(a, own);
            else return next_step<NR>(steps, a);
        };
        while (!lost && next()) {
            const int n = it.n;
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
            int p0 = it.tile * kTile;
            for (int i = 0; i < n; ++i, ++n_tile, p0 += kTile) {
                if (warp == 0) {
                    if (i == 0) ok &= warp_wait(&M->x_full, n_item & 1, fail);
                    ok &= mma.scores(n_tile);
                }
                ok &= warp_wait(&M->s_full, n_tile & 1, fail);
                tc_fence_after();
                float s[NC];
                tmem_ldn<NC>(lanes + TM_S + col0, s);
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
                        if (p0 + p >= M->seen[g][c]) s[c] = -CUDART_INF_F;
                }
                float top = s[0];
#pragma unroll
                for (int c = 1; c < NC; ++c) top = fmaxf(top, s[c]);
                if (bar_any(bar, 128, top > kMoveAt || i == 0 || !ok)) {
                    // a new maximum for every column of the group
                    const float mx = lanes_reduce<NC, true>(s, lane);
                    if (lane < NC) M->red[g][quarter][lane] = mx;
                    if (bar_any(bar, 128, !ok)) { lost = true; break; }
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
                                const uint32_t at = lanes + TM_O + 64 * j + col0 + c0;
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
                uint8_t *dst = sm + F::P + p * 128u;
#pragma unroll
                for (int c = 0; c < NC; c += 8) {
                    float e[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) e[k] = ex2_approx(s[c + k]);
#pragma unroll
                    for (int k = 0; k < 8; k += 2) l[(c + k) / 2] = __fadd2_rn(l[(c + k) / 2], make_float2(e[k], e[k + 1]));
                    *reinterpret_cast<uint4 *>(dst + ((((col0 + c) >> 3) ^ (p & 7)) << 4)) = pack_h8(e);
                }
                tc_fence_before();
                if (!left_out(n_tile)) warp_arrive(&M->p_full);
                if (warp == 0) ok &= mma.output(n_tile, i > 0, i + 1 == n);
            }
            if (lost) break;
            // ---- the row tile's (piece's) output
            const bool whole = it.head && it.tail;
            const int slot = 2 * cta + (it.head ? 1 : 0);      // a piece that starts here goes on behind
            if (n > 0) {
                ok &= warp_wait(&M->o_full, n_item & 1, fail);
                if (bar_any(bar, 128, !ok)) break;
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
                M->f[g][lane] = none ? 0.f : pow2(a.exponent) / sum;
                if (col0 + lane < it.rows) {
                    if (!whole) a.ws_lse[slot * NR + col0 + lane] = lg;
                    else if (a.lse) a.lse[it.row + col0 + lane] = lg * 0.6931471805599453f;
                }
            }
            bar_sync(bar, 128);
            const int rows = it.rows;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                float ov[NC];
                if (n > 0) {
                    tmem_ldn<NC>(lanes + TM_O + 64 * j + col0, ov);
                    tmem_wait_ld();
                }
                const int ch = 128 * j + p;
#pragma unroll
                for (int c = 0; c < NC; ++c) ov[c] = n > 0 ? ov[c] * M->f[g][c] : 0.f;
                if (!whole) {
                    float *dst = a.ws_o + ((size_t)slot * NR + col0) * kLatent + ch;
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (col0 + c < rows) dst[(size_t)c * kLatent] = ov[c];
                } else {
                    // pairs of channels: even lanes store column c, odd lanes column c + 1
                    __nv_bfloat16 *dst = a.o + ((size_t)it.row + col0) * kLatent + (ch & ~1);
                    const bool odd = lane & 1;
#pragma unroll
                    for (int c = 0; c < NC; c += 2) {
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? ov[c] : ov[c + 1], 1);
                        const uint32_t two = odd ? pack_bf2(got, ov[c + 1]) : pack_bf2(ov[c], got);
                        if (col0 + c + odd < rows)
                            *reinterpret_cast<uint32_t *>(dst + (size_t)(c + odd) * kLatent) = two;
                    }
                }
            }
            tc_fence_before();
            // the tile that starts here and goes on: who holds its last piece
            if (t == 0 && it.head && !it.tail) {
                const long long last = it.unit + it.tiles - 1;
                const int blind = min(rows, max(0, (1 - min(1, it.first_tok)) * a.H - it.row_in_seq));
                a.split[cta] = Split{it.row, rows, (int)(last / M->begin.each) - cta / a.side + 1, blind};
            }
        }
        // nothing of this CTA's products is in flight when its TMEM goes
        if (warp == 0) end_products(&M->done, fail);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*fail && t == 0) atomicOr(&g_kda_latent4_decode_error, kErrWait);   // a role gave up
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
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
    a.scale_log2 = scale * 1.4426950408889634f * pow2(a.exponent);
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
