// Attention over the paged cache on the CUDA cores: any element type, head
// size and row count.  float32 calls use it (the tensor cores would round
// their operands).
//
// Per (query, key): x = score(q . k), running maximum m and l = sum 2^(x - m),
// o = sum 2^(x - m) v, one pass over the keys (attention.cuh: the split over
// the grid and the join).  A block holds 16 queries and stages 32 keys at a
// time in shared memory as float32; 8 threads share a query: each scores four
// of the 32 keys and owns D/8 output columns.
//
// Bound by shared-memory reads and FMA issue (per key 2*D FMA for each query),
// not by HBM.
#include "attention.cuh"

namespace specv {
namespace {

constexpr int RT = 16, KT = 32, NT = 128;

template <typename T, int DP> struct SimtSmem {
    float q[RT][DP];
    float k[KT][DP + 4];   // + 4: the eight keys a warp reads lie in different banks
    float v[KT][DP];
    float s[RT][KT + 1];
    float o[RT][DP];
    float m[RT], l[RT];
    int kp[KT];
    int64_t koff[KT];      // element offset of the key's row; -1: none
    AttnRows<RT> rows;
    AttnPlan plan;
    int last;
};

template <typename T, int DP> __global__ void __launch_bounds__(NT) attn_simt_kernel(AttnParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    SimtSmem<T, DP> &sh = *reinterpret_cast<SimtSmem<T, DP> *>(raw);
    constexpr int VEC = Elem<T>::VEC;
    const int tid = threadIdx.x, row = tid >> 3, sub = tid & 7;
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
        float m = -INFINITY, l = 0.0f, o[DP / 8];
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) o[j] = 0.0f;
        const int t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
        const int *table = p.mode == 1 ? p.stable : p.table + (int64_t)it.b * p.max_blocks;
        for (int t = (int)(u - it.u0); t < t1; ++t) {
            const int c0 = it.keys.lo + t * KT, n = min(KT, it.keys.hi - c0);  // n <= 0: no keys
            __syncthreads();
            if (tid < KT) {
                const int c = c0 + tid;
                int64_t off = -1;
                if (tid < n) {
                    if (p.tk && p.mode == 0 && c >= it.keys.len) {
                        off = (int64_t)it.b * p.tsb + ((int64_t)(c - it.keys.len) * p.H + it.h) * p.D;
                    } else {
                        off = entry_offset(p, table, c, it.h);
                        if (off < 0) attn_flag(p, it.b);
                    }
                    sh.kp[tid] = key_position(p, it, c);
                }
                sh.koff[tid] = off;
            }
            __syncthreads();
            for (int i = tid; i < KT * (DP / VEC); i += NT) {
                const int k = i / (DP / VEC), d = (i - k * (DP / VEC)) * VEC;
                const int64_t off = sh.koff[k];
                float x[VEC], y[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[e] = y[e] = 0.0f;
                if (off >= 0 && d < p.D) {
                    const bool cand = p.tk && p.mode == 0 && c0 + k >= it.keys.len;
                    unpack<T>(ld_nc16(static_cast<const T *>(cand ? p.tk : p.kc) + off + d), x);
                    unpack<T>(ld_nc16(static_cast<const T *>(cand ? p.tv : p.vc) + off + d), y);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    sh.k[k][d + e] = x[e];
                    sh.v[k][d + e] = y[e];
                }
            }
            __syncthreads();
            float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int d = 0; d < DP; d += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&sh.q[row][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 b = *reinterpret_cast<const float4 *>(&sh.k[sub + 8 * j][d]);
                    dot[j] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, dot[j]))));
                }
            }
            float mt = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = sub + 8 * j;
                float x = -INFINITY;
                if (sh.koff[k] >= 0) {
                    const int dist = pos_dist(sh.rows.qp[row], sh.kp[k]);
                    if (attn_visible<RT>(p, it, sh.rows, row, c0 + k, sh.kp[k], dist))
                        x = attn_score<sizeof(T) == 4>(dot[j], p.score, sh.rows.slope[row], dist);
                }
                dot[j] = x;
                mt = fmaxf(mt, x);
            }
#pragma unroll
            for (int q = 4; q > 0; q >>= 1) mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, q));
            // the reference m2 = max * log2(e), rounded; weights 2^(x*log2(e) - m2)
            const float m2 = fmaxf(m, mt * kLog2e), ref = m2 == -INFINITY ? 0.0f : m2;
            const float corr = rel_weight(m, ref);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = dot[j] == -INFINITY ? 0.0f : exp2f(fmaf(dot[j], kLog2e, -ref));
                sh.s[row][sub + 8 * j] = e;
                sum += e;
            }
#pragma unroll
            for (int q = 4; q > 0; q >>= 1) sum += __shfl_xor_sync(kFull, sum, q);
            l = l * corr + sum;
            m = m2;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) o[j] *= corr;
#pragma unroll 4
            for (int k = 0; k < KT; ++k) {
                const float w = sh.s[row][k];
                if (w != 0.0f) {  // a masked key's V may hold anything
#pragma unroll
                    for (int j = 0; j < DP / 32; ++j) {
                        const float4 b = *reinterpret_cast<const float4 *>(&sh.v[k][(j * 8 + sub) * 4]);
                        o[4 * j] = fmaf(w, b.x, o[4 * j]);
                        o[4 * j + 1] = fmaf(w, b.y, o[4 * j + 1]);
                        o[4 * j + 2] = fmaf(w, b.z, o[4 * j + 2]);
                        o[4 * j + 3] = fmaf(w, b.w, o[4 * j + 3]);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < DP / 32; ++j)
            *reinterpret_cast<float4 *>(&sh.o[row][(j * 8 + sub) * 4]) = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        if (sub == 0) {
            sh.m[row] = m;
            sh.l[row] = l;
        }
        __syncthreads();
        attn_finish<T, RT, NT>(p, sh.plan, it, sh.rows, &sh.o[0][0], DP, sh.m, sh.l, &sh.last);
        u = it.u0 + it.ntiles;
        if (u >= uend) break;
        it = attn_next(p, it, p.H * rtiles, rtiles, KT);
    }
}

template <typename T, int DP> cudaError_t launch(const AttnParams &p, int sms, cudaStream_t s) {
    const int smem = (int)sizeof(SimtSmem<T, DP>);
    cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = (sms < kAttnSmsMax ? sms : kAttnSmsMax) * (DP == 256 ? 2 : 4);
    attn_simt_kernel<T, DP><<<grid, NT, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_t(const AttnParams &p, int sms, cudaStream_t s) {
    if (p.D <= 64) return launch<T, 64>(p, sms, s);
    if (p.D <= 128) return launch<T, 128>(p, sms, s);
    return launch<T, 256>(p, sms, s);
}

}  // namespace

cudaError_t launch_attn_simt(const AttnParams &p, int dtype, int sms, cudaStream_t s) {
    return dtype == SPEC_DTYPE_BF16 ? launch_t<__nv_bfloat16>(p, sms, s) : launch_t<float>(p, sms, s);
}

}  // namespace specv
