// Tensor-core pieces shared by the latent-attention kernels: TMEM loads and
// stores of other widths, waits that give up together, 2D to 4D bf16 TMA
// maps.
#pragma once

#include <math_constants.h>

#include "latent_common.cuh"
#include "tc_layout.cuh"

namespace kda {
namespace tc {

constexpr float kHuge = 3.402823466e38f;   // the largest finite number

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8p(uint32_t taddr, const float *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}
// N consecutive columns of this thread's lane (N a multiple of 8); the values
// are there after tmem_wait_ld().
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 8) tmem_ld8(taddr + c, v + c);
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const float (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 8) tmem_st8p(taddr + c, v + c);
}

// One lane of a converged warp, the same every time: what it guards is known
// to the compiler as warp-uniform, so descriptors stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
// A shared-memory operand as two words: the low one holds the address (14
// bits of 16 bytes: shared memory ends below 2^18, so offsets add without a
// carry) and the leading offset, the high one is constant over a kernel.  An
// offset costs one 32-bit add, on a path that issues a product every 40 to 80
// cycles.
struct Operand {
    uint32_t lo, hi;
    __device__ __forceinline__ Operand operator+(uint32_t bytes) const { return Operand{lo + (bytes >> 4), hi}; }
};
__device__ __forceinline__ Operand operand(const void *p, uint32_t lbo, uint32_t sbo) {
    const uint64_t d = smem_desc(smem_u32(p), lbo, sbo, kSwizzle128B);
    return Operand{(uint32_t)d, (uint32_t)(d >> 32)};
}
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, Operand a, Operand b, uint32_t idesc, bool acc = true) {
    if (ACC)
        asm volatile(
            "{\n\t.reg .b64 a, b;\n\t.reg .pred p;\n\t"
            "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.eq.u32 p, 0, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
            "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .b64 a, b;\n\t.reg .pred p;\n\t"
            "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
            "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"((uint32_t)acc)
            : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, Operand b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .b64 b;\n\t.reg .pred p;\n\t"
        "mov.b64 b, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

// A bounded wait that also ends when another role of the block has given up.
// The first poll, which is the only one where the wait is over already, is a
// handful of instructions: the MMA warp's time is its instructions'.
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool poll_on(uint32_t bar, uint32_t parity, volatile int *fail) {
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (poll(bar, parity)) return true;
        if ((i & 63u) == 63u && *fail) return false;
    }
    *fail = 1;
    return false;
}
__device__ __forceinline__ bool wait_or_fail(uint32_t bar, uint32_t parity, volatile int *fail) {
    return poll(bar, parity) || poll_on(bar, parity, fail);
}
__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, volatile int *fail) {
    return wait_or_fail(smem_u32(bar), parity, fail);
}
// The same by a whole warp, with one verdict.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *fail) {
    return __all_sync(0xffffffffu, wait_or_fail(bar, parity, fail));
}
// A product warp that has given up goes on to the end of its key tile, but
// releases nothing (the lane that issues asks its own verdict): the copy warp
// would arm a barrier again whose last copy may be on its way.
//
// Ends a block's products before its tensor memory goes (one warp, the one
// that issued them): they need nothing from the other roles, so this waits for
// them whether a role has given up or not.
__device__ __forceinline__ void end_products(uint64_t *done, volatile int *fail) {
    if (elect_one()) mma_commit(done);
    if (!mbar_wait(done, 0, kWaitLimit)) *fail = 1;
    __syncwarp();
}
// Waits for the last copies to each of `bars` barriers that were armed `uses`
// times in turn: a block ends only when nothing is written to its shared
// memory any more.
__device__ __forceinline__ void land(uint64_t *bar, uint32_t uses, uint32_t bars) {
    for (uint32_t i = uses > bars ? uses - bars : 0; i < uses; ++i)
        mbar_wait(bar + i % bars, (i / bars) & 1, kWaitLimit);
}
// A warp's arrival: one for its 32 lanes, after what each of them did.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Debug builds can leave out one arrival, so that a test sees a wait of the
// other roles run out: that of the first block's first softmax warp on the key
// tile (of those it takes) that the host has set; none unless it has.
#ifdef KDA_DEBUG
static __device__ unsigned int g_leave_out = 0xffffffffu;
static inline cudaError_t set_leave_out(unsigned int tile) {   // this translation unit's
    return cudaMemcpyToSymbol(g_leave_out, &tile, sizeof(tile));
}
#endif
__device__ __forceinline__ bool left_out(uint32_t tile) {
#ifdef KDA_DEBUG
    return blockIdx.x == 0 && threadIdx.x < 32 && tile == g_leave_out;
#else
    return false;
#endif
}

// Named barrier over `threads` threads; true if any of them passed `x`.
__device__ __forceinline__ bool bar_any(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// 128B-swizzled map of dense bf16 rows (their number a multiple of 8) as
// [8-row group][64-column block][row][column]: boxes of box_blocks column
// blocks x box_groups groups, which lie in shared memory as [group][block][8
// rows][128 B].  One copy brings several column blocks of a page; groups are
// box_blocks KB apart, blocks 1 KB, in both operand readings.
inline bool make_map_groups(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, uint32_t box_blocks,
                            uint32_t box_groups) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {64, 8, (cuuint64_t)(cols / 64), (cuuint64_t)(rows / 8)};
    cuuint64_t strides[3] = {(cuuint64_t)cols * 2, 128, (cuuint64_t)cols * 16};
    cuuint32_t box[4] = {64, 8, box_blocks, box_groups};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 128B-swizzled maps of bf16 rows: boxes of 64 columns x box_rows rows.
inline bool make_map_rows(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t stride,
                          uint32_t box_rows) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// ... of a [T, H, cols] tensor: boxes of 64 columns x 1 head x box_rows tokens.
inline bool make_map_heads(CUtensorMap *m, const void *base, int64_t cols, int64_t H, int64_t T,
                           uint32_t box_rows) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)H, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)(H * cols) * 2};
    cuuint32_t box[3] = {64, 1, box_rows};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- launches that follow one another closely
// A kernel launched with launch_early may begin once every block of the one
// before it in the stream has called let_next_begin() or ended; it must call
// wait_for_previous(), which returns when that one is complete and its writes
// are visible, before it touches any global memory.  What it does before that
// (barriers, tensor memory) runs under the other's end.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                         A &&...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// ---- host: a kernel's shared-memory limit and the device's SM count
// Both cost a driver call of a microsecond or so; they hold for a device's
// context, so they are asked for and set once in each (`id` of cuCtxGetId
// tells a context made by a device reset from the one before it).
struct KernelSetup {
    static constexpr int kDevices = 64;
    std::mutex mu;
    unsigned long long ctx[kDevices] = {};
    int sms[kDevices] = {};

    cudaError_t get(const void *kernel, int smem_bytes, int *n_sms) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lk(mu);
        unsigned long long id = context_id();
        if (id == 0 || id != ctx[dev]) {
            e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
            if (e != cudaSuccess) return e;
            ctx[dev] = context_id();
        }
        *n_sms = sms[dev];
        return cudaSuccess;
    }
    static unsigned long long context_id() {
        static PFN_cuCtxGetId_v12000 fn = [] {
            cudaDriverEntryPointQueryResult q;
            void *p = nullptr;
            if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
                q != cudaDriverEntryPointSuccess)
                p = nullptr;
            return reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
        }();
        unsigned long long id = 0;
        return fn && fn(nullptr, &id) == CUDA_SUCCESS ? id : 0;
    }
};

}  // namespace tc
}  // namespace kda
