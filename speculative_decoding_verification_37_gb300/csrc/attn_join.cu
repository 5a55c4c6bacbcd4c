// The join of items whose keys were split over several blocks (attention.cuh),
// as a kernel of its own: one row of blocks per block of the attention kernel, for
// the item that begins in it and goes on in others; a warp per query.
// A programmatic dependent of the attention kernel.
#include "attention.cuh"
#include "tma.cuh"

namespace specv {
namespace {

constexpr int kWarps = 8;

template <typename T> __global__ void __launch_bounds__(32 * kWarps, 4) attn_join_kernel(AttnParams p, int rt_rows) {
    // what comes next may start once every block here has
    pdl_launch_dependents();
    pdl_wait_primary();
    const SplitItem it = p.split[blockIdx.x];
    if (it.blocks < 2) return;
    const int per = p.S * p.G;
    const int64_t nrows = p.mode == 1 ? (int64_t)p.B * per : per;
    for (int r = blockIdx.y * kWarps + (threadIdx.x >> 5); r < rt_rows; r += gridDim.y * kWarps) {
        const int64_t k = (int64_t)it.rt * rt_rows + r;
        if (k >= nrows) return;
        const int b = p.mode == 1 ? (int)(k / per) : it.b, q = (int)(k - (p.mode == 1 ? (int64_t)b * per : 0));
        const int s = q / p.G;
        attn_join_row<T, 4>(p, it.ok, rt_rows, blockIdx.x, it.blocks, r,
                            ((int64_t)b * p.S + s) * p.Hq + it.h * p.G + (q - s * p.G));
    }
}

}  // namespace

cudaError_t launch_attn_join(const AttnParams &p, int rt_rows, int blocks, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)((rt_rows + kWarps * 4 - 1) / (kWarps * 4)));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<__nv_bfloat16>, p, rt_rows);
}

}  // namespace specv
