// The attention weight cached entries accumulate (spec_attention_weights).
//
// weight[c] += sum over the committed candidates j with c <= e_j and the query
// heads h of exp(x(j, h, c) - lse(j, h)).  The softmax's sum is known, so no
// pass over the values and no second pass is needed: K is read once.  A tile
// is 64 entries of one request with all its cached heads, so one thread owns
// an entry's whole sum: nothing is added atomically and the result does not
// depend on timing.
#include "attention.cuh"

namespace specv {
namespace {

constexpr int KT = 64, NT = 128, RQ = 16;  // entries per tile, queries staged at a time

template <typename T, int DP> struct WSmem {
    float k[KT][DP + 4];
    float q[RQ][DP];
    float part[KT];
    int64_t koff[KT];
    int kp[KT];
    int qp[RQ], own[RQ], first;   // position, own entry (-1: no such query)
    float slope[RQ], lse2[RQ];
    AttnPlan plan;
};

// CUDA-core version: any element type.  Two threads share an entry, each
// taking half the queries.
template <typename T, int DP> __global__ void __launch_bounds__(NT) weights_simt_kernel(WeightsParams wp) {
    extern __shared__ __align__(16) unsigned char raw[];
    WSmem<T, DP> &sh = *reinterpret_cast<WSmem<T, DP> *>(raw);
    const AttnParams &p = wp.a;
    constexpr int VEC = Elem<T>::VEC;
    const int tid = threadIdx.x, key = tid & (KT - 1), half = tid / KT;
    attn_plan<NT>(p, sh.plan, 1, KT);
    int64_t u = (int64_t)blockIdx.x * sh.plan.share;
    const int64_t uend = min(sh.plan.total, u + sh.plan.share);
    if (u >= uend) return;
    AttnItem it = attn_find<NT>(p, sh.plan, u, 1, 1, KT);
    while (true) {
        const int b = it.b, n = it.keys.ok ? p.n_slots[b] : 0;
        const int *slots = p.slots ? p.slots + (int64_t)b * p.slots_stride : nullptr;
        bool bad = !it.keys.ok;
        for (int j = tid; slots && j < n; j += NT) bad = bad || slots[j] < 0 || slots[j] >= p.S;
        const bool skip = __syncthreads_or(bad);
        if (skip && u == it.u0 && tid == 0) attn_flag(p, b);
        const int t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0), rows = n * p.G;
        const int first = p.first ? p.first[b] : (int)0x80000000;
        for (int t = (int)(u - it.u0); t < t1 && !skip; ++t) {
            const int c0 = it.keys.lo + t * KT, nk = min(KT, it.keys.hi - c0);
            if (nk <= 0) break;
            const int cand0 = it.keys.len - n;  // the candidates' first entry
            __syncthreads();
            if (tid < KT) {
                const int c = c0 + tid;
                int64_t off = -1;
                int kp = 0;
                if (tid < nk) {
                    off = entry_offset(p, p.table + (int64_t)b * p.max_blocks, c, 0);
                    if (off < 0) attn_flag(p, b);
                    kp = p.key_pos && c < cand0 ? p.key_pos[(int64_t)b * p.kps + c] : c;
                    if (c >= cand0 && p.pos) kp = p.pos[(int64_t)b * p.S + (slots ? slots[c - cand0] : c - cand0)];
                }
                sh.koff[tid] = off;
                sh.kp[tid] = kp;
            }
            float acc = 0.0f;
            for (int h = 0; h < p.H; ++h) {
                __syncthreads();
                for (int i = tid; i < KT * (DP / VEC); i += NT) {
                    const int k = i / (DP / VEC), d = (i - k * (DP / VEC)) * VEC;
                    float x[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) x[e] = 0.0f;
                    if (sh.koff[k] >= 0 && d < p.D)
                        unpack<T>(ld_nc16(static_cast<const T *>(p.kc) + sh.koff[k] + (int64_t)h * p.D + d), x);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) sh.k[k][d + e] = x[e];
                }
                for (int r0 = 0; r0 < rows; r0 += RQ) {
                    __syncthreads();
                    if (tid < RQ) {
                        const int r = r0 + tid;
                        sh.own[tid] = -1;
                        if (r < rows) {
                            const int j = r / p.G, s = slots ? slots[j] : j, hq = h * p.G + r - j * p.G;
                            const float lse = wp.lse_in[((int64_t)b * p.S + s) * p.Hq + hq];
                            sh.own[tid] = lse == -INFINITY ? -1 : cand0 + j;
                            sh.lse2[tid] = lse * kLog2e;
                            sh.qp[tid] = p.pos ? p.pos[(int64_t)b * p.S + s] : cand0 + j;
                            sh.slope[tid] = p.slopes ? p.slopes[hq] : 0.0f;
                        }
                    }
                    for (int i = tid; i < RQ * DP; i += NT) {
                        const int k = i / DP, d = i - k * DP, r = r0 + k;
                        float x = 0.0f;
                        if (r < rows && d < p.D) {
                            const int j = r / p.G, s = slots ? slots[j] : j;
                            x = to_f32(static_cast<const T *>(p.q)[b * p.qsb + s * p.qss + (h * p.G + r - j * p.G) * p.qsh + d]);
                        }
                        sh.q[k][d] = x;
                    }
                    __syncthreads();
#pragma unroll
                    for (int g = 0; g < RQ / 8; ++g) {
                        const int q0 = half * (RQ / 2) + g * 4;
                        float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                        for (int d = 0; d < DP; d += 4) {
                            const float4 a = *reinterpret_cast<const float4 *>(&sh.k[key][d]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float4 q = *reinterpret_cast<const float4 *>(&sh.q[q0 + j][d]);
                                dot[j] = fmaf(a.x, q.x, fmaf(a.y, q.y, fmaf(a.z, q.z, fmaf(a.w, q.w, dot[j]))));
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int q = q0 + j, c = c0 + key;
                            if (sh.koff[key] < 0 || c > sh.own[q]) continue;
                            const int dist = pos_dist(sh.qp[q], sh.kp[key]);
                            if (sh.kp[key] < first || (p.window > 0 && dist >= p.window)) continue;
                            acc += exp2f(fmaf(attn_score<sizeof(T) == 4>(dot[j], p.score, sh.slope[q], dist), kLog2e, -sh.lse2[q]));
                        }
                    }
                }
            }
            if (half == 1) sh.part[key] = acc;
            __syncthreads();
            if (half == 0 && key < nk && sh.koff[key] >= 0) {
                const int c = c0 + key;
                wp.weight[b * wp.wstride + c] += acc + sh.part[key];
            }
            if (half == 1 && key < nk && wp.key_pos_out && c0 + key >= cand0)
                wp.key_pos_out[(int64_t)b * p.kps + c0 + key] = sh.kp[key];
        }
        u = it.u0 + it.ntiles;
        if (u >= uend) break;
        it = attn_next(p, it, 1, 1, KT);
    }
}

template <typename T, int DP> cudaError_t launch(const WeightsParams &p, int sms, cudaStream_t s) {
    const int smem = (int)sizeof(WSmem<T, DP>);
    cudaError_t e = cudaFuncSetAttribute(weights_simt_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    weights_simt_kernel<T, DP><<<sms * (DP == 256 ? 2 : 4), NT, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_t(const WeightsParams &p, int sms, cudaStream_t s) {
    if (p.a.D <= 64) return launch<T, 64>(p, sms, s);
    if (p.a.D <= 128) return launch<T, 128>(p, sms, s);
    return launch<T, 256>(p, sms, s);
}

}  // namespace

cudaError_t launch_weights_simt(const WeightsParams &p, int dtype, int sms, cudaStream_t s) {
    return dtype == SPEC_DTYPE_BF16 ? launch_t<__nv_bfloat16>(p, sms, s) : launch_t<float>(p, sms, s);
}

}  // namespace specv
