// The fifth-generation tensor cores and TMA tiles of a page's rows, for the
// kernels that read the paged cache in boxes (attn_tc.cu, attn_weights_tc.cu).
#pragma once

#include <cuda.h>

#include "attention.cuh"
#include "tma.cuh"

namespace specv {
namespace {

// ---- tcgen05 -------------------------------------------------------------
__device__ __forceinline__ void tc_alloc(uint32_t *dst) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t t) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(unsigned long long *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// D (TMEM) (+)= A (shared) B (shared)^T
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// D (TMEM) (+)= A (TMEM) B (shared)
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
#define R8(x, i) "=f"(x[i]), "=f"(x[i + 1]), "=f"(x[i + 2]), "=f"(x[i + 3]), "=f"(x[i + 4]), "=f"(x[i + 5]), "=f"(x[i + 6]), "=f"(x[i + 7])
#define W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// 32 columns of this thread's lane
__device__ __forceinline__ void tc_ld32(float *x, uint32_t t) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : R8(x, 0), R8(x, 8), R8(x, 16), R8(x, 24)
        : "r"(t));
}
template <int N> __device__ __forceinline__ void tc_ldx(float *x, uint32_t t) {
#pragma unroll
    for (int i = 0; i < N; i += 32) tc_ld32(x + i, t + i);
}
template <int N> __device__ __forceinline__ float max_of(const float *x) {
    float a = x[0], b = x[1], c = x[2], d = x[3];
#pragma unroll
    for (int i = 4; i < N; i += 4) {
        a = fmaxf(a, x[i]);
        b = fmaxf(b, x[i + 1]);
        c = fmaxf(c, x[i + 2]);
        d = fmaxf(d, x[i + 3]);
    }
    return fmaxf(fmaxf(a, b), fmaxf(c, d));
}
__device__ __forceinline__ void tc_ld16(float *x, uint32_t t) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : R8(x, 0), R8(x, 8)
                 : "r"(t));
}
__device__ __forceinline__ void tc_ld8(float *x, uint32_t t) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : R8(x, 0) : "r"(t));
}
__device__ __forceinline__ void tc_st16(uint32_t t, const uint32_t *x) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        W8(x, 0), W8(x, 8)
        : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t t, const uint32_t *x) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
        W8(x, 0), W8(x, 8), W8(x, 16), W8(x, 24)
        : "memory");
}
#undef R8
#undef W8

// Shared-memory operand, 128-byte swizzle (8 rows of 128 bytes an atom): lbo /
// sbo are the byte steps described at the uses.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// bf16 x bf16 -> f32, M = 128; bn: B's rows (N) are contiguous
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool bn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (bn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap *m, int x, int y, int z, unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap *m, int x, int y, int z, int w,
                                     unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma5(uint32_t dst, const CUtensorMap *m, int x, int y, int z, int w, int v,
                                     unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
            dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned long long *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) { return __vcmpeq2(x & 0x7f807f80u, 0x7f807f80u); }

// barriers of n threads under an id of their own
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// ---- host ------------------------------------------------------------------
using TcEncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline TcEncodeFn tc_encode_fn() {
    static const TcEncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<TcEncodeFn>(f);
    }();
    return fn;
}

inline bool tc_encode(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return tc_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box,
                       ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A tile of 128 keys in shared memory: atoms of 8 rows x 128 bytes (64 columns).
// Heads of 128 come whole, a box of a page's rows a copy, the halves of their
// columns next to each other; others a half a copy, zeros past their columns, and
// then all rows of the second half behind those of the first.
// (WH: whole; constants, because sums put together at run time cost heads of 128
// 1 to 2%.)
template <int NH, bool WH> struct TcLayout {
    static constexpr uint32_t group = NH == 2 && WH ? 2048 : 1024;  // bytes from 8 rows to the next 8
    static constexpr uint32_t half = NH == 2 && WH ? 1024 : 128 * 128;  // from a half to the other
};
// One box: p.box rows of head h from row r on.
template <int NH, bool WH>
__device__ __forceinline__ void tc_copy_box(uint32_t dst, const CUtensorMap *m, int r, int h, unsigned long long *bar) {
    if (NH == 2 && WH) {
        tma5(dst, m, 0, 0, 0, r >> 3, h, bar);
    } else {
        tma3(dst, m, 0, h, r, bar);
        if (NH == 2) tma3(dst + TcLayout<NH, WH>::half, m, 64, h, r, bar);
    }
}

// The layer's K and V planes, a box of p.box rows of one cached head a copy.
inline bool tc_cache_map(const AttnParams &p, CUtensorMap *cm) {
    const cuuint64_t row = (cuuint64_t)p.H * p.D * 2, rows = (cuuint64_t)(2 * p.nb * p.bs);
    if (p.D == 128) {  // [row group][half of the columns][8 rows][64 columns]: a page's rows in one copy
        const cuuint64_t dims[5] = {64, 8, 2, rows / 8, (cuuint64_t)p.H}, strides[4] = {row, 128, 8 * row, 256};
        const cuuint32_t box[5] = {64, 8, 2, (cuuint32_t)p.box / 8, 1};
        return tc_encode(cm, p.kc, 5, dims, strides, box);
    } else {
        const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.H, rows}, strides[2] = {(cuuint64_t)p.D * 2, row};
        const cuuint32_t box[3] = {64, 1, (cuuint32_t)p.box};
        return tc_encode(cm, p.kc, 3, dims, strides, box);
    }
}

}  // namespace
}  // namespace specv
