// Causal attention of many new tokens with expanded keys and values, on the
// tensor cores: the prefill side of latent attention.
//
// Head h of token j has the key [kv[j][h][0:128] | k_pe[j]] and the value
// kv[j][h][128:256]; the last 64 key channels are one row a token for all
// heads and are read as such.  The queries of a sequence are its last tokens:
// query i of nq sees keys 0 .. nk - nq + i.
//   s = scale <q, k>,   o = softmax(s) v,   lse = ln sum e^s
//
// A work tile is 256 queries of one (sequence, head).  The grid has a CTA for
// each; a CTA (one fits an SM) that is done with one takes over the next that
// has not been launched, so its loads and products follow on without a gap.
// It runs over the keys 128 at a time, with two halves of 128 queries in
// turn on the tensor cores, so that one half's products cover the other's
// softmax:
//   S_g [128 x 128] = Q_g K^T         12 K-steps, Q_g and K from shared memory
//   O_g [128 x 128] += P_g V          8 K-steps, P_g (bf16) from TMEM, in S_g's place
// A softmax thread owns a query: it keeps the row's maximum m, sum and nothing
// else; p = exp2(s scale log2 e - m) with the m of the tile before, and only
// when a score passes m by more than 8 (a factor 256, which fp32 sums and bf16
// probabilities hold without loss) does the row take a new maximum, is O_g
// rescaled in TMEM and the tile's p computed again.  p is rounded to bf16, the
// product's operand type, after the fp32 sum has taken it: 2^-8 of each weight at
// most, independent of the others', beside the bf16 output's own rounding
// (against 64 bits 1.9e-3 to 2.3e-3 in the 2-norm; the output's rounding alone
// makes 1.6e-3 to 1.7e-3).
//
// Few work tiles over many keys (a short chunk behind a long context) would
// leave SMs idle: then the keys of each are cut into pieces, each a work tile
// of its own that leaves its normalised output in fp32 with its log2-sum-exp
// in the workspace, and a second kernel joins them.
//
// Roles: two groups of four softmax warps, an MMA warp, a copy warp that
// feeds a ring of eight 16 KB slots (three a key tile, two a value tile: 1.6
// tiles in flight).  TMEM: S_0, S_1, O_0, O_1, 128 columns each.
//
// What bounds it: the products with what shares their memories.  A key tile
// takes both halves 3,600 cycles: 2,560 of multiply-adds (a step of S reads both
// operands from shared memory at its full rate, so the copies' 80 KB delay it:
// 2,660), the scores' and weights' way out of and into TMEM beside the
// accumulators, and the waits between a half's product and its next scores; the
// softmax (1,200 cycles a half) hides under the other half.  (Handing P over in
// two halves of 64 keys, so that P V begins earlier, changed nothing: 394 us.)
// Measured: 4,096 tokens at 96 heads 392 us (1.32 PFLOP/s of the causal
// multiply-adds, 70 % of the measured dense rate); 1,024 and 1,000 tokens
// behind 8,192 at 32 heads 286 us (67 %: 256 equal work tiles on 152 SMs, two
// rounds).
#include <algorithm>
#include <type_traits>

#include "latent_tc.cuh"

namespace kda {

using namespace tc;

// Error word of this file's kernel (bit 0: a bounded wait gave up, or
// cu_seqlens broke its precondition).
__device__ unsigned int g_kda_latent_prefill_error = 0;

namespace {

constexpr int kThreads = 320;             // 8 softmax warps, the MMA warp, the copy warp
constexpr int kHalf = 128;                // queries a half
constexpr int kTileQ = 2 * kHalf;
constexpr int kTileK = 128;
constexpr int kSms = 152;                 // the device's, for the host's choice of pieces
constexpr int kMaxPieces = 32;            // a lane each in the joining kernel
constexpr int kSlots = 8;
constexpr uint32_t kSlot = 16384;
constexpr uint32_t SM_Q = 0;              // [2 halves][3 blocks of 64 channels][128 rows x 128 B]
constexpr uint32_t SM_RING = 6 * 16384;
constexpr uint32_t SM_MISC = SM_RING + kSlots * kSlot;
constexpr float kMoveAt = 8.f;            // log2 of the factor a score may pass the maximum by
constexpr uint32_t TM_S = 0, TM_O = 256;
// Keys and values of the heads listed together: what stays in L2 (4,096 tokens
// at 96 heads: 376 us; one head at a time 393, all of them 404).
constexpr int64_t kL2Bytes = 48 << 20;

struct Work {
    int valid;                            // 0: there is none
    int h, q0, k0, nk;                    // head; first token of the sequence's queries; of its keys, and keys
    int i0;                               // first query of the tile
    int rows[2];                          // queries of each half
    int lo;                               // first key tile of this piece
    int n[2];                             // key tiles of it that each half sees any of
    int piece;
    int first;                            // keys that the sequence's query 0 sees (may be <= 0)
};

struct Misc {
    uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2];   // by key tile, even and odd
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], done;
    uint64_t answer_full, work_full[2], work_empty[2];
    alignas(16) uint4 answer;             // to the request for a further work tile
    Work work[2];                         // the copy warp's, for the other roles
    uint32_t tmem;
    int fail;
    uint32_t n_q[2], n_k, n_v, asked;     // copies and further work tiles asked for, by barrier
    int tiles;                            // work tiles of all sequences (of one head)
    long long warp_sum[kThreads / 32];
    int ahead[kThreads];                  // work tiles before thread t's sequences
};
constexpr uint32_t SM_BYTES = SM_MISC + sizeof(Misc);
static_assert(SM_BYTES + 1024 <= 232448, "shared memory of an SM");

struct Args {
    const int32_t *cu_q, *cu_k;
    int N, Tq, Tk, H;
    bool causal;
    int heads_together;                   // heads whose work tiles are listed together
    int most;                             // work tiles of one head that valid offsets can give
    int pieces;                           // of a work tile's keys; 1: not cut
    float *ws_lse, *ws_o;                 // pieces' log2-sum-exp [pieces][Tq * H], outputs [pieces][Tq * H][128]
    bool o_aligned32;
    float scale_log2;                     // scale * log2 e
    __nv_bfloat16 *o;
    float *lse;
};

__device__ __forceinline__ int queries_of(const Args &a, int b, bool flag) {
    const int t0 = a.cu_q[b], t1 = a.cu_q[b + 1];
    const bool bad = t0 < 0 || t1 < t0 || t1 > a.Tq;
    if (flag) {
        const int k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
        if (bad || k0 < 0 || k1 < k0 || k1 > a.Tk) atomicOr(&g_kda_latent_prefill_error, kErrWait);
    }
    return bad ? 0 : t1 - t0;
}

// First token of sequence b's keys, and keys (none of a range that leaves [0, Tk]).
__device__ __forceinline__ void keys_of(const Args &a, int b, int &k0, int &nk) {
    k0 = a.cu_k[b];
    nk = a.cu_k[b + 1] - k0;
    if (k0 < 0 || nk < 0 || k0 > a.Tk - nk) k0 = nk = 0;
}

// Work tile `id` of the grid.  Heads are listed in groups whose keys and
// values fit in L2 together; in a group, the packed queries' tiles from the last
// to the first: within a sequence what is handed out last sees the fewest keys.
// (Over several the order is the batch's: a long sequence that comes first in it
// is begun last.)
__device__ __forceinline__ void get_work(const Args &a, const Misc *M, int id, Work &w) {
    const int tiles = M->tiles;
    w.valid = id >= 0 && (unsigned)id / a.pieces < (unsigned)tiles * (unsigned)a.H;
    if (!w.valid) return;
    w.piece = id % a.pieces;
    id /= a.pieces;
    const unsigned group = (unsigned)id / ((unsigned)tiles * a.heads_together);
    const int h0 = group * a.heads_together, heads = min(a.heads_together, a.H - h0);
    const int in = (int)((unsigned)id - group * tiles * a.heads_together);
    w.h = h0 + in % heads;
    int k = tiles - 1 - in / heads;
    // the thread whose sequences hold tile k, then the sequence
    int lo = 0, hi = kThreads;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (M->ahead[mid] <= k) lo = mid;
        else hi = mid;
    }
    k -= M->ahead[lo];
    const int per = (a.N + kThreads - 1) / kThreads;
    int b = lo * per, nq = queries_of(a, b, false);
    while (k >= (nq + kTileQ - 1) / kTileQ) {
        k -= (nq + kTileQ - 1) / kTileQ;
        nq = queries_of(a, ++b, false);
    }
    w.q0 = a.cu_q[b];
    keys_of(a, b, w.k0, w.nk);
    w.i0 = k * kTileQ;
    w.first = w.nk - nq + 1;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        w.rows[g] = max(0, min(kHalf, nq - w.i0 - g * kHalf));
        const int sees = a.causal ? max(0, w.first + w.i0 + g * kHalf + w.rows[g] - 1) : w.nk;
        w.n[g] = w.rows[g] > 0 ? (sees + kTileK - 1) / kTileK : 0;
    }
    // this piece's share of the key tiles
    const int n = max(w.n[0], w.n[1]);
    w.lo = (int)((int64_t)n * w.piece / a.pieces);
    const int end = (int)((int64_t)n * (w.piece + 1) / a.pieces);
#pragma unroll
    for (int g = 0; g < 2; ++g) w.n[g] = max(0, min(w.n[g], end) - w.lo);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Asks for a work tile that no CTA has begun: the grid has a CTA for each, and
// a running one takes over the next that has not been launched.  The answer
// (16 bytes) comes to shared memory like a copy.
__device__ __forceinline__ void ask_work(uint4 *answer, uint64_t *bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
}
// The block index taken over, or -1 (none was left).
__device__ __forceinline__ int taken_work(const uint4 *answer) {
    uint32_t ok, x = 0;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return ok ? (int)x : -1;
}
// The other roles' walk over the CTA's work tiles, by whole warps: the copy
// warp finds out what they are (a search and a few dependent loads, 2,500
// cycles) while the tile before is computed.
struct Tiles {
    uint32_t r = 0;
    __device__ __forceinline__ bool next(Misc *M, Work &w, bool &ok, volatile int *fail) {
        const uint32_t at = r & 1;
        ok = __all_sync(0xffffffffu, ok) && warp_wait(&M->work_full[at], (r >> 1) & 1, fail);
        if (!ok) return false;
        w = M->work[at];
        warp_arrive(&M->work_empty[at]);
        ++r;
        return w.valid;
    }
};

__device__ __forceinline__ void st_global32(void *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_pe,
                      const Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Misc *M = reinterpret_cast<Misc *>(sm + SM_MISC);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

    // ---- barriers and tensor memory, under the end of the kernel before this one
    if (t == 0) {
        M->fail = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&M->k_full[i], 1);
            mbar_init(&M->v_full[i], 1);
            mbar_init(&M->k_empty[i], 1);
            mbar_init(&M->v_empty[i], 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&M->q_full[g], 1);
            mbar_init(&M->q_empty[g], 1);
            mbar_init(&M->s_full[g], 1);
            mbar_init(&M->p_full[g], 4);      // warps of a group
            mbar_init(&M->o_full[g], 1);
        }
        mbar_init(&M->done, 1);
        mbar_init(&M->answer_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&M->work_full[i], 1);
            mbar_init(&M->work_empty[i], kThreads / 32 - 1);
        }
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&M->tmem, 512);
    if (warp == 9 && lane == 0) {
        prefetch_tmap(&map_q);
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
        prefetch_tmap(&map_pe);
    }
    wait_for_previous();
    // ---- work tiles ahead of each thread's sequences
    {
        const int per = (a.N + kThreads - 1) / kThreads;
        const int b_lo = min(a.N, t * per), b_hi = min(a.N, b_lo + per);
        long long mine = 0;               // overlapping offsets can give more than 32 bits hold
        for (int b = b_lo; b < b_hi; ++b)
            mine += (queries_of(a, b, blockIdx.x == 0) + kTileQ - 1) / kTileQ;   // CTA 0 flags broken offsets
        long long incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) M->warp_sum[warp] = incl;
        __syncthreads();
        long long before = incl - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += M->warp_sum[w];
            total += M->warp_sum[w];
        }
        M->ahead[t] = (int)before;
        if (t == 0) M->tiles = total > a.most ? 0 : (int)total;   // broken offsets (flagged): no work
    }
    if (a.pieces > 1) let_next_begin();   // the joining kernel (another prefill's blocks would take SMs from this one's)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;
    volatile int *fail = &M->fail;
    Work w;

    if (warp == 9) {
        // ================================================= copies
        // Key tile u fills ring slots 5 u .. 5 u + 2, its value tile 5 u + 3 and 5 u + 4 (modulo 8).
        // The key slots were last the third of key tile u - 2 and both of its value tile, the value
        // slots the first two of key tile u - 1; the MMA warp releases in the order of u.
        uint32_t u = 0;                           // key tiles asked for
        uint32_t n_v = 0, asked = 0, told = 0;    // value tiles, further work tiles, work tiles
        uint32_t n_q[2] = {0, 0};                 // query halves
        bool ok = true;
        auto tell = [&](const Work &x) {          // the other roles, of a work tile (or that none is left)
            const uint32_t at = told & 1;
            if (told >= 2) ok = ok && warp_wait(&M->work_empty[at], ((told >> 1) - 1) & 1, fail);
            if (!ok) return;
            ++told;
            if (lane == 0) {
                M->work[at] = x;
                mbar_arrive(&M->work_full[at]);
            }
            __syncwarp();
            // its queries toward L2 while the tile before still holds their place
            if (x.valid && lane < 6 && (lane < 3 ? x.n[0] : x.n[1]) > 0)
                tma_prefetch_l2_3d(&map_q, 64 * (lane % 3), x.h, x.q0 + x.i0 + (lane / 3) * kHalf);
            __syncwarp();
        };
        get_work(a, M, (int)blockIdx.x, w);
        tell(w);
        while (ok && w.valid) {
            // The next work tile is asked for four key tiles before the end and known two before it:
            // early enough for its first copies, late enough that a block with a long tile does not
            // hold one back that another could begin.
            Work next;
            auto ask = [&]() {
                if (lane == 0) ask_work(&M->answer, &M->answer_full);
                ++asked;
                __syncwarp();
            };
            auto learn = [&]() {
                ok = ok && warp_wait(&M->answer_full, (asked - 1) & 1, fail);
                if (!ok) return;
                get_work(a, M, taken_work(&M->answer), next);
                fence_proxy_async_smem();         // read before the next answer is written there
                __syncwarp();
                tell(next);
            };
            const int n = max(w.n[0], w.n[1]);
            if (n == 0) {
                ask();
                learn();
            }
            // half g's queries, once the tile before is done with theirs
            auto queries = [&](int g) {
                if (w.n[g] == 0) return;
                if (n_q[g] > 0) ok = ok && warp_wait(&M->q_empty[g], (n_q[g] - 1) & 1, fail);
                if (!ok) return;
                ++n_q[g];
                if (lane == 0) {
                    mbar_arrive_expect_tx(&M->q_full[g], 3 * kSlot);
                    for (int c = 0; c < 3; ++c)
                        tma_load_3d(sm + SM_Q + (3 * g + c) * kSlot, &map_q, &M->q_full[g], 64 * c, w.h,
                                    w.q0 + w.i0 + g * kHalf);
                }
                __syncwarp();
            };
            if (n > 0) queries(0);
            for (int i = 0; ok && i < n; ++i) {
                const int tok = w.k0 + (w.lo + i) * kTileK;
                auto slot = [&](int c) { return sm + SM_RING + ((5 * n_v + c) % kSlots) * kSlot; };
                if (u >= 2) ok = warp_wait(&M->v_empty[u & 1], ((u >> 1) - 1) & 1, fail);
                if (!ok) break;
                if (lane == 0) {
                    uint64_t *bar = &M->k_full[u & 1];
                    mbar_arrive_expect_tx(bar, 3 * kSlot);
                    tma_load_3d(slot(0), &map_k, bar, 0, w.h, tok);
                    tma_load_3d(slot(1), &map_k, bar, 64, w.h, tok);
                    tma_load_2d(slot(2), &map_pe, bar, 0, tok);
                }
                __syncwarp();
                ++u;
                if (i == 0) queries(1);
                if (!ok) break;
                if (n_v >= 1) ok = warp_wait(&M->k_empty[(n_v - 1) & 1], ((n_v - 1) >> 1) & 1, fail);
                if (!ok) break;
                if (lane == 0) {
                    uint64_t *bar = &M->v_full[n_v & 1];
                    mbar_arrive_expect_tx(bar, 2 * kSlot);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tma_load_3d(slot(3 + c), &map_v, bar, 128, w.h, tok + 64 * c);
                        tma_load_3d(slot(3 + c) + 8192, &map_v, bar, 192, w.h, tok + 64 * c);
                    }
                }
                __syncwarp();
                ++n_v;
                if (i == max(0, n - 4)) ask();
                if (i == max(0, n - 2)) learn();
            }
            w = next;
        }
        if (lane == 0) {
            M->n_q[0] = n_q[0];
            M->n_q[1] = n_q[1];
            M->n_k = u;
            M->n_v = n_v;
            M->asked = asked;
        }
    } else if (warp == 8) {
        // ================================================= matrix products
        // The whole warp walks and waits, one lane issues.
        constexpr uint32_t id_s = instr_desc(kFmtBF16, 128, 128, 0, 0);
        constexpr uint32_t id_o = instr_desc(kFmtBF16, 128, 128, 0, 1);
        const Operand q_op = operand(sm + SM_Q, 16, 1024), k_op = operand(sm + SM_RING, 16, 1024);
        const Operand v_op = operand(sm + SM_RING, 8192, 1024);
        const uint32_t k_full = smem_u32(M->k_full), v_full = smem_u32(M->v_full);
        const uint32_t k_empty = smem_u32(M->k_empty), v_empty = smem_u32(M->v_empty);
        const uint32_t s_full = smem_u32(M->s_full), p_full = smem_u32(M->p_full), o_full = smem_u32(M->o_full);
        const uint32_t q_full = smem_u32(M->q_full), q_empty = smem_u32(M->q_empty);
        uint32_t u = 0, cnt0 = 0, cnt1 = 0;               // key tiles, tiles of each half
        uint32_t nq0 = 0, nq1 = 0;                        // query halves
        bool ok = true;
        auto scores = [&](int g, uint32_t tile) {         // one lane
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const Operand k = k_op + ((5 * tile + c) % kSlots) * kSlot, q = q_op + (3 * g + c) * kSlot;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (c == 0 && e == 0) mma_ss<false>(tmem + TM_S + 128 * g, q, k, id_s, false);
                    else mma_ss<true>(tmem + TM_S + 128 * g, q + e * 32u, k + e * 32u, id_s);
                }
            }
            commit(s_full + 8 * g);
        };
        auto product = [&](int g, uint32_t tile, bool acc) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const Operand v = v_op + ((5 * tile + 3 + c) % kSlots) * kSlot;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mma_ts(tmem + TM_O + 128 * g, tmem + TM_S + 128 * g + 32 * c + 8 * e, v + e * 2048u, id_o,
                           acc || c > 0 || e > 0);
            }
        };
        // half 0's first scores of a work tile, whose first key tile is `tile`
        auto first_scores = [&](int n0, uint32_t tile) {
            ok &= wait_or_fail(q_full, nq0++ & 1, fail);
            ok &= wait_or_fail(k_full + 8 * (tile & 1), (tile >> 1) & 1, fail);
            tc_fence_after();
            if (elect_one()) {
                scores(0, tile);
                if (n0 == 1 && ok) commit(q_empty);
            }
            __syncwarp();
        };
        Tiles tiles;
        bool more = tiles.next(M, w, ok, fail), begun = false;
        while (more && __all_sync(0xffffffffu, ok)) {
            const int n0 = w.n[0], n1 = w.n[1], n = max(n0, n1);
            if (n == 0) {
                more = tiles.next(M, w, ok, fail);
                continue;
            }
            if (n0 > 0 && !begun) first_scores(n0, u);
            begun = false;
            if (n1 > 0) ok &= wait_or_fail(q_full + 8, nq1++ & 1, fail);
            ok &= wait_or_fail(k_full + 8 * (u & 1), (u >> 1) & 1, fail);
            tc_fence_after();
            if (elect_one()) {
                if (n1 > 0) scores(1, u);
                if (n1 == 1 && ok) commit(q_empty + 8);
                if (ok) commit(k_empty + 8 * (u & 1));
            }
            __syncwarp();
            for (int i = 0; i < n; ++i, ++u) {
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                const uint32_t x = u + 1;
                // half 0: its product, then its next scores (which follow the product in the pipe:
                // it reads P in their place); then half 1
                ok &= wait_or_fail(v_full + 8 * (u & 1), (u >> 1) & 1, fail);
                if (i < n0) ok &= wait_or_fail(p_full, cnt0++ & 1, fail);
                tc_fence_after();
                if (i < n0 && elect_one()) {
                    product(0, u, i > 0);
                    if (i + 1 == n0) commit(o_full);
                }
                __syncwarp();
                if (i + 1 < n) {
                    ok &= wait_or_fail(k_full + 8 * (x & 1), (x >> 1) & 1, fail);
                    tc_fence_after();
                    if (i + 1 < n0 && elect_one()) {
                        scores(0, x);
                        if (i + 2 == n0 && ok) commit(q_empty);
                    }
                    __syncwarp();
                } else {
                    // the last key tile: half 0 begins the next work tile while half 1 ends this one
                    more = tiles.next(M, w, ok, fail);
                    if (more && w.n[0] > 0) {
                        first_scores(w.n[0], x);
                        begun = true;
                    }
                }
                if (i < n1) ok &= wait_or_fail(p_full + 8, cnt1++ & 1, fail);
                tc_fence_after();
                if (elect_one()) {
                    if (i < n1) {
                        product(1, u, i > 0);
                        if (i + 1 == n1) commit(o_full + 8);
                    }
                    if (ok) commit(v_empty + 8 * (u & 1));
                    if (i + 1 < n1) scores(1, x);
                    if (i + 2 == n1 && ok) commit(q_empty + 8);
                    if (i + 1 < n && ok) commit(k_empty + 8 * (x & 1));
                }
                __syncwarp();
            }
        }
        // nothing of this CTA's products is in flight when its TMEM goes
        end_products(&M->done, fail);
    } else {
        // ================================================= softmax, output
        const int g = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;              // query of the half
        const uint32_t base = tmem + ((uint32_t)quarter << 21);
        const uint32_t ts = base + TM_S + 128 * g, to = base + TM_O + 128 * g;
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
        uint32_t cnt = 0, n_out = 0, u = 0;
        bool ok = true;
        Tiles tiles;
        while (ok && tiles.next(M, w, ok, fail)) {
            const int rows = g ? w.rows[1] : w.rows[0], n = g ? w.n[1] : w.n[0];
            const int n_all = max(w.n[0], w.n[1]);
            if (rows == 0) { u += n_all; continue; }
            const int i_row = w.i0 + g * kHalf + row;     // query of the sequence
            // keys that the row sees, and those that all rows of the warp see, from the piece's first on
            const int from_key = w.lo * kTileK;
            const int sees = (a.causal ? min(w.nk, w.first + i_row) : w.nk) - from_key;
            const int all_see = (a.causal ? min(w.nk, w.first + w.i0 + g * kHalf + quarter * 32) : w.nk) - from_key;
            const int nk = w.nk - from_key;
            float neg_m = 0.f, l = 0.f;
            for (int i = 0; i < n; ++i, ++cnt) {
                const int lim = sees - i * kTileK;        // columns from here on are masked
                const bool masked = all_see - i * kTileK < kTileK;
                ok = warp_wait(&M->s_full[g], cnt & 1, fail);
                if (!ok) break;
                tc_fence_after();
                uint32_t p[64];
                float top, sum;
                // p and their sum from the row's present maximum; the largest exponent
                auto weights = [&](auto with_mask) {
                    constexpr bool kMask = decltype(with_mask)::value;
                    const float2 nm2 = make_float2(neg_m, neg_m);
                    float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
                    float tp = -CUDART_INF_F;
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t s[32];
                        tmem_ld32(ts + 32 * ch, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float2 d = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, nm2);
                            if (kMask) {
                                if (32 * ch + c >= lim) d.x = -CUDART_INF_F;
                                if (32 * ch + c + 1 >= lim) d.y = -CUDART_INF_F;
                            }
                            tp = fmaxf(tp, fmaxf(d.x, d.y));
                            const float2 e = make_float2(ex2_approx(d.x), ex2_approx(d.y));
                            if (c & 2) acc1 = __fadd2_rn(acc1, e);
                            else acc0 = __fadd2_rn(acc0, e);
                            p[16 * ch + c / 2] = pack_bf2(e.x, e.y);
                        }
                    }
                    top = tp;
                    sum = (acc0.x + acc0.y) + (acc1.x + acc1.y);
                };
                // a new maximum: in the first tile the tile's own, later only a larger one (and O
                // and the sum are rescaled).  A row that sees nothing in the first tile sees
                // nothing at all
                auto move = [&]() {
                    float mx = -CUDART_INF_F;
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t s[32];
                        tmem_ld32(ts + 32 * ch, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float d = fmaf(__uint_as_float(s[c]), a.scale_log2, neg_m);
                            mx = fmaxf(mx, masked && 32 * ch + c >= lim ? -CUDART_INF_F : d);
                        }
                    }
                    float up = i > 0 ? fmaxf(mx, 0.f) : mx == -CUDART_INF_F ? 0.f : mx;
                    const float now = neg_m - up;
                    up = neg_m - now;                      // what the rounded maximum really moves by
                    neg_m = now;
                    if (i > 0) {                           // the products before this tile are done (s_full)
                        const float f = ex2_approx(-up);
                        l *= f;
#pragma unroll 1
                        for (int c0 = 0; c0 < 128; c0 += 16) {
                            float ov[16];
                            tmem_ld16(to + c0, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; ++c) ov[c] *= f;
                            tmem_st16(to + c0, ov);
                        }
                        tmem_wait_st();
                    }
                };
                auto weigh = [&]() {
                    if (masked) weights(std::true_type{});
                    else weights(std::false_type{});
                };
                if (i == 0) {
                    // a first maximum from 32 of the columns: the others seldom pass it by kMoveAt.
                    // A row that sees none of them sees nothing
                    uint32_t s[32];
                    tmem_ld32(ts, s);
                    tmem_wait_ld();
                    float mx = -CUDART_INF_F;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        mx = fmaxf(mx, c >= lim ? -CUDART_INF_F : __uint_as_float(s[c]) * a.scale_log2);
                    neg_m = mx == -CUDART_INF_F ? 0.f : -mx;
                }
                weigh();
                // (lanes behind the half's queries hold another sequence's, or what no sequence
                // has: they have no say)
                if (__any_sync(0xffffffffu, top > kMoveAt && row < rows)) {
                    move();
                    weigh();
                }
                l += sum;
#pragma unroll
                for (int c = 0; c < 64; c += 16) tmem_st16u(ts + c, p + c);
                if ((i + 1) * kTileK > nk) {
                    // value rows behind the sequence's end are its neighbour's: they must not meet
                    // a zero weight
                    const uint32_t first = 5 * (u + i) + 3;
                    ok = warp_wait(&M->v_full[(u + i) & 1], ((u + i) >> 1) & 1, fail);
                    const int from = nk - i * kTileK;
                    for (int e = row; ok && e < (kTileK - from) * 16; e += kHalf) {
                        const int rr = from + (e >> 4), ch = e & 15;
                        *reinterpret_cast<uint4 *>(sm + SM_RING + ((first + (rr >> 6)) % kSlots) * kSlot +
                                                   (ch >> 3) * 8192u + (rr & 63) * 128u + (ch & 7) * 16u) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                if (!left_out(cnt)) warp_arrive(&M->p_full[g]);
                if (!ok) break;
            }
            u += n_all;
            if (!ok) break;
            // ---- output
            if (n > 0) {
                ok = warp_wait(&M->o_full[g], n_out & 1, fail);
                if (!ok) break;
                ++n_out;
                tc_fence_after();
            }
            // A row that sees nothing has o = 0; one that sees keys has 1 / l, NaN included, and 0 / 0
            // where each of its scores is -inf.  A piece may be without weight: the joining kernel tells
            const bool none = a.pieces > 1 ? l == 0.f : sees <= 0;
            const float inv = none ? 0.f : 1.f / l;
            const float lg = none ? -CUDART_INF_F : log2f(l) - neg_m;
            const size_t out = ((size_t)w.q0 + i_row) * a.H + w.h;
            const size_t at = (size_t)w.piece * a.Tq * a.H + out;   // in the workspace
#pragma unroll
            for (int c0 = 0; c0 < 128; c0 += 32) {
                uint32_t ov[32] = {};
                if (n > 0) {
                    tmem_ld32(to + c0, ov);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) ov[c] = none ? 0u : __float_as_uint(__uint_as_float(ov[c]) * inv);
                if (row < rows) {
                    // a lane stores its own row: whole 32-byte sectors halve the store unit's work
                    if (a.pieces > 1) {
#pragma unroll
                        for (int c = 0; c < 32; c += 8)
                            st_global32(a.ws_o + at * 128 + c0 + c, ov + c);
                    } else {
                        __nv_bfloat16 *dst = a.o + out * 128 + c0;
#pragma unroll
                        for (int c = 0; c < 32; c += 16) {
                            uint32_t x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                x[e] = pack_bf2(__uint_as_float(ov[c + 2 * e]), __uint_as_float(ov[c + 2 * e + 1]));
                            if (a.o_aligned32) {
                                st_global32(dst + c, x);
                            } else {
                                *reinterpret_cast<uint4 *>(dst + c) = make_uint4(x[0], x[1], x[2], x[3]);
                                *reinterpret_cast<uint4 *>(dst + c + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                            }
                        }
                    }
                }
            }
            if (row < rows) {
                if (a.pieces > 1) a.ws_lse[at] = lg;
                else if (a.lse) a.lse[out] = lg * 0.6931471805599453f;
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*fail) {                          // a role gave up: nobody may have waited for the last copies
        if (t == 0) atomicOr(&g_kda_latent_prefill_error, kErrWait);
        if (warp == 9) {
            land(&M->q_full[0], M->n_q[0], 1);
            land(&M->q_full[1], M->n_q[1], 1);
            land(M->k_full, M->n_k, 2);
            land(M->v_full, M->n_v, 2);
            land(&M->answer_full, M->asked, 1);
        }
    }
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// Joins the pieces of every row, o = sum_k 2^(lse_k - lse) o_k in the order of
// the keys: a warp a row, four channels a lane.
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads)
latent_prefill_join_kernel(const Args a) {
    const int64_t rows = (int64_t)a.Tq * a.H;
    const int64_t r = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    let_next_begin();
    wait_for_previous();                      // the pieces are written
    const int tok = (int)min(r / a.H, (int64_t)a.Tq - 1), b = seq_of_token(a.cu_q, a.N, tok);
    if (r >= rows || b < 0) return;           // behind the last sequence
    float v = lane < a.pieces ? a.ws_lse[lane * rows + r] : -CUDART_INF_F;
    float mx = fmaxf(v, -kHuge);              // finite, so that no weight is -inf - -inf
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    v = ex2_approx(v - mx);
    float sum = v;                            // NaN where a piece's is
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    float inv = 1.f / sum;
    if (sum == 0.f) {                         // the row sees nothing (0), or only scores of -inf (0 / 0)
        int k0, nk;
        keys_of(a, b, k0, nk);
        if ((a.causal ? nk - (a.cu_q[b + 1] - tok) + 1 : nk) <= 0) inv = 0.f;
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < a.pieces; ++k) {
        const float f = __shfl_sync(0xffffffffu, v, k) * inv;
        const float4 x = reinterpret_cast<const float4 *>(a.ws_o + (k * rows + r) * 128)[lane];
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
    }
    reinterpret_cast<uint2 *>(a.o + r * 128)[lane] = make_uint2(pack_bf2(acc.x, acc.y), pack_bf2(acc.z, acc.w));
    if (a.lse && lane == 0) a.lse[r] = (mx + log2f(sum)) * 0.6931471805599453f;
}

// Work tiles there can be at most: n queries of a sequence are at most
// (n - 1) / 256 + 1 tiles.
int64_t most_tiles(int N, int64_t Tq, int H) {
    const int64_t seqs = std::min<int64_t>(N, Tq);        // with queries
    return ((Tq - seqs) / kTileQ + seqs) * H;
}

// Pieces that a work tile's keys are cut into: those with the least time by
// this count, in key tiles (1.9 us) of the average sequence.  The SMs take the
// pieces in rounds, a piece costs 2.5 key tiles beside its own (first loads,
// first softmax, output); joining costs three (its launch) and its pieces'
// 131 KB written and read.  Measured against one piece, us a call: 1 head, 100
// queries behind 4,000: 17 / 54; 256 behind 20,000: 25 / 283; 8 heads, 1,024
// behind 8,192: 60 / 137; 2 heads, 4,096: 29 / 62; and where the count keeps
// one: 16 heads, 300 behind 300: 16, two pieces 19.  The host knows the average
// alone: one long context among short ones is cut too little or not at all.  16
// heads, 15 queries behind 300 each and 512 behind 65,536: one piece, 970 us (an
// even share of the SMs would be 210); 8 chunks of 256, one of them behind
// 100,000: three pieces, 535 us (160).
int pieces_of(int N, int64_t Tq, int64_t Tk, int H) {
    const int64_t tiles = most_tiles(N, Tq, H);
    const double keys = (double)((Tk / N + kTileK - 1) / kTileK);
    if (tiles > 2 * kSms) return 1;
    int best = 1;
    double least = 0;
    for (int k = 1; k <= kMaxPieces && (k == 1 || 2 * k <= keys); ++k) {
        const double rounds = (double)((tiles * k + kSms - 1) / kSms);
        const double cost = rounds * (keys / k + 2.5) + (k > 1 ? 3 + 0.024 * tiles * k : 0);
        if (k == 1 || cost < least) {
            best = k;
            least = cost;
        }
    }
    return best;
}

}  // namespace

// Workspace of a call that cuts its keys: the pieces' outputs, then their
// log2-sum-exp.
size_t latent_prefill_workspace_bytes(int N, int64_t Tq, int64_t Tk, int H) {
    const int pieces = pieces_of(N, Tq, Tk, H);
    return pieces > 1 ? (size_t)pieces * Tq * H * 129 * sizeof(float) : 0;
}

cudaError_t launch_latent_prefill(const void *q, const void *kv, const void *k_pe, int64_t pe_stride,
                                  const int32_t *cu_q, const int32_t *cu_k, float scale, bool causal,
                                  void *o, float *lse, int N, int64_t Tq, int64_t Tk, int H, void *ws,
                                  cudaStream_t stream) {
    static KernelSetup setup;
    int sms = 0;                          // not needed: the grid is the work's
    cudaError_t e = setup.get(reinterpret_cast<const void *>(latent_prefill_kernel), SM_BYTES + 1024, &sms);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv, mp;
    if (!make_map_heads(&mq, q, 192, H, Tq, kHalf)) return cudaErrorInvalidValue;
    mk = mv = mp = mq;                    // without keys none of the others is read through
    if (Tk > 0 && (!make_map_heads(&mk, kv, 256, H, Tk, kTileK) || !make_map_heads(&mv, kv, 256, H, Tk, 64) ||
                   !make_map_rows(&mp, k_pe, 64, Tk, pe_stride, kTileK)))
        return cudaErrorInvalidValue;
    const int together = (int)std::min<int64_t>(H, std::max<int64_t>(1, kL2Bytes / (std::max<int64_t>(Tk, 1) * 512)));
    Args a;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.N = N;
    a.Tq = (int)Tq;
    a.Tk = (int)Tk;
    a.H = H;
    a.causal = causal;
    a.heads_together = together;
    a.most = (int)most_tiles(N, Tq, 1);
    a.pieces = pieces_of(N, Tq, Tk, H);
    a.ws_o = static_cast<float *>(ws);
    a.ws_lse = a.pieces > 1 ? a.ws_o + (size_t)a.pieces * Tq * H * 128 : nullptr;
    a.o_aligned32 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    // a CTA for each piece of each work tile there can be
    e = launch_early(latent_prefill_kernel, (unsigned)(most_tiles(N, Tq, H) * a.pieces), kThreads, SM_BYTES + 1024,
                     stream, mq, mk, mv, mp, a);
    if (e != cudaSuccess || a.pieces == 1) return e;
    return launch_early(latent_prefill_join_kernel,
                        (unsigned)((Tq * H + kJoinThreads / 32 - 1) / (kJoinThreads / 32)), kJoinThreads, 0, stream, a);
}

cudaError_t read_latent_prefill_error(unsigned int *code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kda_latent_prefill_error, sizeof(unsigned int));
    if (e != cudaSuccess || !reset) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kda_latent_prefill_error, &zero, sizeof(unsigned int));
}

#ifdef KDA_DEBUG
cudaError_t latent_prefill_leave_out(unsigned int tile) { return set_leave_out(tile); }
#endif

}  // namespace kda
