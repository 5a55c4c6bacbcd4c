// Attention over the paged cache on the CUDA cores, for float32 (the tensor cores
// would round its operands).
//
// Per (query, key): x = score(q . k), running maximum m and l = sum 2^(x - m),
// o = sum 2^(x - m) v, one pass over the keys (attention.cuh: the split over
// the grid and the join).  A block holds 16 R queries and stages 32 keys at a
// time in shared memory as float32; 8 threads share R queries: each scores four
// of the 32 keys and owns D/8 output columns for each of them.
//
// Bound by shared-memory reads and FMA issue (per key 2*D FMA for each query),
// not by HBM: R = 4 reads 8 times 16 bytes for 64 FMA where R = 1 reads 5 for
// 16.  Few queries take R = 1, whose blocks are smaller and more.  8 requests of
// 15 queries on up to 777 entries of 2 heads of 72: 27.6 us in a graph.
#include "attention.cuh"
#include "tma.cuh"

namespace specv {
namespace {

constexpr int KT = 32, NT = 128;

// 16 bytes, or zeros where `bytes` is 0
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T, int DP, int RT> struct SimtSmem {
    float q[RT][DP];
    float k[KT][DP + 4];   // + 4: the eight keys a warp reads lie in different banks
    float v[KT][DP];
    float s[RT][KT + 1];
    float o[RT][DP];
    float m[RT], l[RT];
    int kp[2][KT];         // two tiles' keys: position,
    int64_t koff[2][KT];   // element offset of the row; -1: none
    AttnRows<RT> rows;
    AttnPlan plan;
    int last;
};

template <typename T, int DP, int R>
__global__ void __launch_bounds__(NT, DP == 256 || R == 4 ? 2 : 4) attn_simt_kernel(AttnParams p) {
    constexpr int RT = 16 * R;
    extern __shared__ __align__(16) unsigned char raw[];
    SimtSmem<T, DP, RT> &sh = *reinterpret_cast<SimtSmem<T, DP, RT> *>(raw);
    static_assert(sizeof(T) == 4, "rows are copied as they are");
    const int tid = threadIdx.x, row0 = tid >> 3, sub = tid & 7;  // rows row0, row0 + 16, ...
    const int per = p.S * p.G;
    const int64_t nrows = p.mode == 1 ? (int64_t)p.B * per : per;
    const int rtiles = (int)((nrows + RT - 1) / RT);
    attn_plan<NT>(p, sh.plan, p.H * rtiles, KT);
    int64_t u = (int64_t)blockIdx.x * sh.plan.share;
    const int64_t uend = min(sh.plan.total, u + sh.plan.share);
    if (u >= uend) return;
    AttnItem it = attn_find<NT>(p, sh.plan, u, p.H * rtiles, rtiles, KT);
    while (true) {
        attn_rows<RT, NT>(p, it, sh.rows, tid);
        __syncthreads();
        for (int i = tid; i < RT * DP; i += NT) {
            const int r = i / DP, d = i - r * DP;
            sh.q[r][d] = sh.rows.q[r] >= 0 && d < p.D ? to_f32(static_cast<const T *>(p.q)[sh.rows.q[r] + d]) : 0.0f;
        }
        if (!it.keys.ok && u == it.u0 && it.h == 0 && it.rt == 0 && tid == 0) attn_flag(p, it.b);
        float m[R], l[R], o[R][DP / 8];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) o[r][j] = 0.0f;
        }
        const int t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
        const int *table = p.mode == 1 ? p.stable : p.table + (int64_t)it.b * p.max_blocks;
        const int t0 = (int)(u - it.u0);
        // this thread's key of a tile (the first KT threads)
        int64_t off_next = -1;
        int kp_next = 0;
        auto look_up = [&](int t) {
            const int c = it.keys.lo + t * KT + tid;
            off_next = -1;
            if (tid >= KT || c >= it.keys.hi) return;
            if (p.tk && p.mode == 0 && c >= it.keys.len) {
                off_next = (int64_t)it.b * p.tsb + ((int64_t)(c - it.keys.len) * p.H + it.h) * p.D;
            } else {
                off_next = entry_offset(p, table, c, it.h);
                if (off_next < 0) attn_flag(p, it.b);
            }
            kp_next = key_position(p, it, c);
        };
        auto keep = [&](int t) {
            if (tid < KT) {
                sh.koff[t & 1][tid] = off_next;
                sh.kp[t & 1][tid] = kp_next;
            }
        };
        auto copy = [&](int t, bool v) {  // a tile's K or V rows, zeros where there is none
            for (int i = tid; i < KT * (DP / 4); i += NT) {
                const int k = i / (DP / 4), d = (i - k * (DP / 4)) * 4;
                const int64_t off = sh.koff[t & 1][k];
                const bool in = off >= 0 && d < p.D, cand = p.tk && p.mode == 0 && it.keys.lo + t * KT + k >= it.keys.len;
                const T *from = static_cast<const T *>(v ? (cand ? p.tv : p.vc) : (cand ? p.tk : p.kc));
                cp_async16(smem_u32(v ? &sh.v[k][d] : &sh.k[k][d]), in ? from + off + d : from, in ? 16 : 0);
            }
        };
        look_up(t0);
        keep(t0);
        __syncthreads();
        copy(t0, false);
        cp_async_wait_all();
        __syncthreads();
        // V arrives while the scores are taken, the next K during the rest
        for (int t = t0; t < t1; ++t) {
            const int c0 = it.keys.lo + t * KT;
            const int *s_kp = sh.kp[t & 1];
            const int64_t *s_koff = sh.koff[t & 1];
            if (t + 1 < t1) look_up(t + 1);
            copy(t, true);
            float dot[R][4];
#pragma unroll
            for (int r = 0; r < R; ++r) dot[r][0] = dot[r][1] = dot[r][2] = dot[r][3] = 0.0f;
#pragma unroll 4
            for (int d = 0; d < DP; d += 4) {
                float4 a[R];
#pragma unroll
                for (int r = 0; r < R; ++r) a[r] = *reinterpret_cast<const float4 *>(&sh.q[row0 + 16 * r][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 b = *reinterpret_cast<const float4 *>(&sh.k[sub + 8 * j][d]);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        dot[r][j] = fmaf(a[r].x, b.x, fmaf(a[r].y, b.y, fmaf(a[r].z, b.z, fmaf(a[r].w, b.w, dot[r][j]))));
                }
            }
            if (t + 1 < t1) keep(t + 1);
            cp_async_wait_all();
            __syncthreads();
            if (t + 1 < t1) copy(t + 1, false);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = row0 + 16 * r;
                float mt = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = sub + 8 * j;
                    float x = -INFINITY;
                    if (s_koff[k] >= 0) {
                        const int dist = pos_dist(sh.rows.qp[row], s_kp[k]);
                        if (attn_visible<RT>(p, it, sh.rows, row, c0 + k, s_kp[k], dist))
                            x = attn_score<sizeof(T) == 4>(dot[r][j], p.score, sh.rows.slope[row], dist);
                    }
                    dot[r][j] = x;
                    mt = fmaxf(mt, x);
                }
#pragma unroll
                for (int q = 4; q > 0; q >>= 1) mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, q));
                // the reference m2 = max * log2(e), rounded; weights 2^(x*log2(e) - m2)
                const float m2 = fmaxf(m[r], mt * kLog2e), ref = m2 == -INFINITY ? 0.0f : m2;
                const float corr = rel_weight(m[r], ref);
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = dot[r][j] == -INFINITY ? 0.0f : exp2f(fmaf(dot[r][j], kLog2e, -ref));
                    sh.s[row][sub + 8 * j] = e;
                    sum += e;
                }
#pragma unroll
                for (int q = 4; q > 0; q >>= 1) sum += __shfl_xor_sync(kFull, sum, q);
                l[r] = l[r] * corr + sum;
                m[r] = m2;
#pragma unroll
                for (int j = 0; j < DP / 8; ++j) o[r][j] *= corr;
            }
            __syncwarp();
#pragma unroll 4
            for (int k = 0; k < KT; ++k) {
                float w[R];
#pragma unroll
                for (int r = 0; r < R; ++r) w[r] = sh.s[row0 + 16 * r][k];
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) {
                    const float4 b = *reinterpret_cast<const float4 *>(&sh.v[k][(j * 8 + sub) * 4]);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (w[r] != 0.0f) {  // a masked key's V may hold anything
                            o[r][4 * j] = fmaf(w[r], b.x, o[r][4 * j]);
                            o[r][4 * j + 1] = fmaf(w[r], b.y, o[r][4 * j + 1]);
                            o[r][4 * j + 2] = fmaf(w[r], b.z, o[r][4 * j + 2]);
                            o[r][4 * j + 3] = fmaf(w[r], b.w, o[r][4 * j + 3]);
                        }
                }
            }
            cp_async_wait_all();
            __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = row0 + 16 * r;
#pragma unroll
            for (int j = 0; j < DP / 32; ++j)
                *reinterpret_cast<float4 *>(&sh.o[row][(j * 8 + sub) * 4]) =
                    make_float4(o[r][4 * j], o[r][4 * j + 1], o[r][4 * j + 2], o[r][4 * j + 3]);
            if (sub == 0) {
                sh.m[row] = m[r];
                sh.l[row] = l[r];
            }
        }
        __syncthreads();
        attn_finish<T, RT, NT>(p, sh.plan, it, sh.rows, &sh.o[0][0], DP, sh.m, sh.l, &sh.last);
        u = it.u0 + it.ntiles;
        if (u >= uend) break;
        it = attn_next(p, it, p.H * rtiles, rtiles, KT);
    }
}

template <typename T, int DP, int R> cudaError_t launch(const AttnParams &p, int sms, cudaStream_t s) {
    const int smem = (int)sizeof(SimtSmem<T, DP, 16 * R>);
    cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<T, DP, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // (at most 8 / R blocks an SM: the workspace's partial results)
    const int grid = (sms < kAttnSmsMax ? sms : kAttnSmsMax) * (DP == 256 || R == 4 ? 2 : 4);
    attn_simt_kernel<T, DP, R><<<grid, NT, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int DP> cudaError_t launch_r(const AttnParams &p, int sms, cudaStream_t s) {
    const int64_t rows = p.mode == 1 ? (int64_t)p.B * p.S * p.G : (int64_t)p.S * p.G;
    if (rows <= 16) return launch<T, DP, 1>(p, sms, s);
    if (rows <= 32 || DP == 256) return launch<T, DP, 2>(p, sms, s);
    return launch<T, DP, DP == 256 ? 2 : 4>(p, sms, s);
}

template <typename T> cudaError_t launch_t(const AttnParams &p, int sms, cudaStream_t s) {
    if (p.D <= 64) return launch_r<T, 64>(p, sms, s);
    if (p.D <= 128) return launch_r<T, 128>(p, sms, s);
    return launch_r<T, 256>(p, sms, s);
}

}  // namespace

cudaError_t launch_attn_simt(const AttnParams &p, int sms, cudaStream_t s) {
    return launch_t<float>(p, sms, s);
}

}  // namespace specv
