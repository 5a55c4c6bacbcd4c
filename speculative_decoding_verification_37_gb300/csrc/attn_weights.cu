// The attention weight cached entries accumulate (spec_attention_weights).
//
// weight[c] += sum over the committed candidates j with c <= e_j and the query
// heads h of exp(x(j, h, c) - lse(j, h)).  The softmax's sum is known, so no
// pass over the values and no second pass is needed: K is read once.  A tile
// is 32 or 128 entries of one request with all its cached heads, so an entry's sum
// stays in one block: nothing is added atomically and the result does not
// depend on timing.
#include "attention.cuh"
#include "tma.cuh"

namespace specv {
namespace {

constexpr int KT = 32, NT = 128, RQ = 16;  // entries per tile, queries staged at a time

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Out of line: inline it took registers from the loops (f32, 64 requests of 2,048
// entries: 625 us, so 550).
__device__ __noinline__ void shared_positions_call(const WeightsParams &wp, const AttnItem &it, int tid, int nt) {
    shared_positions(wp, it, tid, nt);
}

template <typename T, int DP> struct WSmem {
    float k[2][KT][DP + 4];  // this head's and the next one's
    float q[RQ][DP];
    float part[NT / KT][KT];
    int64_t koff[KT];
    int kp[KT];
    int qp[RQ], own[RQ], first;   // position, own entry (-1: no such query)
    float slope[RQ], lse2[RQ];
    AttnPlan plan;
};

// CUDA-core version: any element type.  A lane has an entry, a warp a quarter of
// the queries, whose elements are broadcast; the next head's rows are copied
// while this one's scores are taken.  Bound by issue and by the queries' staging
// for each head and 16 of them (f32, 64 requests of 2,048 entries, 8 heads of 128:
// up to 5 x 4 queries a head 550 us, up to 4 of them 298, 1.8 TB/s; all of a
// head's rows before its scores, two lanes an entry: 788 and 530).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {  // zeros where `bytes` is 0
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T, int DP> __global__ void __launch_bounds__(NT) weights_simt_kernel(WeightsParams wp) {
    extern __shared__ __align__(16) unsigned char raw[];
    WSmem<T, DP> &sh = *reinterpret_cast<WSmem<T, DP> *>(raw);
    const AttnParams &p = wp.a;
    constexpr int VEC = Elem<T>::VEC;
    const int tid = threadIdx.x, key = tid & (KT - 1), part = tid / KT;
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
        if (!skip && u == it.u0) shared_positions_call(wp, it, tid, NT);
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
            auto copy = [&](int h) {
                for (int i = tid; i < KT * (DP / VEC); i += NT) {
                    const int k = i / (DP / VEC), d = (i - k * (DP / VEC)) * VEC;
                    const bool in = sh.koff[k] >= 0 && d < p.D;
                    const T *from = static_cast<const T *>(p.kc) + (in ? sh.koff[k] + (int64_t)h * p.D + d : 0);
                    float *to = &sh.k[h & 1][k][d];
                    if constexpr (sizeof(T) == 4) {
                        cp_async16(smem_u32(to), from, in ? 16 : 0);
                    } else {
                        float x[VEC];
#pragma unroll
                        for (int e = 0; e < VEC; ++e) x[e] = 0.0f;
                        if (in) unpack<T>(ld_nc16(from), x);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) to[e] = x[e];
                    }
                }
            };
            __syncthreads();
            copy(0);
            for (int h = 0; h < p.H; ++h) {
                cp_async_wait_all();
                __syncthreads();  // this head's rows are there, the last one's done with
                if (h + 1 < p.H) copy(h + 1);
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
#pragma unroll
                    for (int i = tid; i < RQ * (DP / VEC); i += NT) {
                        const int k = i / (DP / VEC), d = (i - k * (DP / VEC)) * VEC, r = r0 + k;
                        float x[VEC];
#pragma unroll
                        for (int e = 0; e < VEC; ++e) x[e] = 0.0f;
                        if (r < rows && d < p.D) {
                            const int j = r / p.G, s = slots ? slots[j] : j;
                            unpack<T>(ld_nc16(static_cast<const T *>(p.q) + b * p.qsb + s * p.qss + (h * p.G + r - j * p.G) * p.qsh + d), x);
                        }
#pragma unroll
                        for (int e = 0; e < VEC; ++e) sh.q[k][d + e] = x[e];
                    }
                    __syncthreads();
                    const int q0 = part * (RQ / (NT / KT));
                    float dot[4] = {0.f, 0.f, 0.f, 0.f};
                    static_assert(RQ == 4 * (NT / KT), "four queries a thread");
#pragma unroll 4
                    for (int d = 0; d < DP; d += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(&sh.k[h & 1][key][d]);
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
            sh.part[part][key] = acc;
            __syncthreads();
            if (part == 0 && key < nk && sh.koff[key] >= 0) {
#pragma unroll
                for (int q = 1; q < NT / KT; ++q) acc += sh.part[q][key];
                wp.weight[b * wp.wstride + c0 + key] += acc;
            }
            if (part == 1 && key < nk && wp.key_pos_out && c0 + key >= cand0)
                wp.key_pos_out[(int64_t)b * p.kps + c0 + key] = sh.kp[key];
        }
        u = it.u0 + it.ntiles;
        if (u >= uend) break;
        it = attn_next(p, it, 1, 1, KT);
    }
}

// bf16 version, on the warp tensor instructions, for the head and page sizes
// that attn_weights_tc.cu does not take.  Bound by latency: the registers that
// hold K leave 16 warps an SM (512 ragged requests of up to 4,096 entries, 8
// heads of 128, capped and biased: 729 us with pages of 4, 3.0 TB/s, 706 of 16,
// which take 394 there).
//
// A warp owns 16 entries of a tile for all cached heads: the entries' K rows are
// the rows (M = 16) of its products, the queries the columns (N = 8).  The order
// in which the products run over the head's columns is free as long as both
// operands share it, so a lane's operand registers are four neighbouring pairs,
// one 16-byte load of its row (and of the query's): K goes from memory straight
// to registers, a head ahead of the arithmetic.  The queries of a request (all
// heads) lie in shared memory.  A lane ends up with two entries and two queries
// of each product, so an entry's sum is local but for three neighbours.
constexpr int WM = 8, WKT = 16 * WM, WNT = 32 * WM;  // warps, entries of a tile, threads
constexpr int kQueryBytes = 80 * 1024;               // shared memory for queries

template <int DP> struct WRow {
    static constexpr int kPitch = DP * 2 + 16;
};

template <int DP> __global__ void __launch_bounds__(WNT, DP == 256 ? 1 : 2) weights_mma_kernel(WeightsParams wp, int per_pass) {
    using T = __nv_bfloat16;
    constexpr int PITCH = WRow<DP>::kPitch, NB = DP / 32;
    extern __shared__ __align__(16) unsigned char raw[];
    const AttnParams &p = wp.a;
    // [queries: head, row][pitch], then per query -lse (log2 units; -inf for none
    // that counts), slope, position, own entry
    const int rows_max = (per_pass * p.G + 7) / 8 * 8, nq = p.H * rows_max;
    unsigned char *sq = raw;
    float4 *s_info = reinterpret_cast<float4 *>(raw + (size_t)nq * PITCH);
    float *s_nlse = reinterpret_cast<float *>(s_info + nq);  // the first of them again, closer together
    __shared__ AttnPlan plan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
    attn_plan<WNT>(p, plan, 1, WKT);
    int64_t u = (int64_t)blockIdx.x * plan.share;
    const int64_t uend = min(plan.total, u + plan.share);
    if (u >= uend) return;
    AttnItem it = attn_find<WNT>(p, plan, u, 1, 1, WKT);
    while (true) {
        const int b = it.b, n = it.keys.ok ? p.n_slots[b] : 0;
        const int *slots = p.slots ? p.slots + (int64_t)b * p.slots_stride : nullptr;
        bool bad = !it.keys.ok;
        for (int j = tid; slots && j < n; j += WNT) bad = bad || slots[j] < 0 || slots[j] >= p.S;
        const bool skip = __syncthreads_or(bad);
        if (skip && u == it.u0 && tid == 0) attn_flag(p, b);
        if (!skip && u == it.u0) shared_positions_call(wp, it, tid, WNT);
        const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
        const int first = p.first ? p.first[b] : (int)0x80000000;
        const int cand0 = it.keys.len - n;  // the candidates' first entry
        const int *table = p.table + (int64_t)b * p.max_blocks;
        for (int j0 = 0; j0 < n && !skip && it.keys.lo < it.keys.hi; j0 += per_pass) {
            const int nj = min(per_pass, n - j0), rows = nj * p.G, rp = (rows + 7) / 8 * 8;
            __syncthreads();
            bool none = false;  // a query that adds nothing
            for (int i = tid; i < p.H * rp; i += WNT) {
                const int h = i / rp, r = i - h * rp, j = j0 + r / p.G, hq = h * p.G + r % p.G;
                int own = -1, qp = 0;
                float nlse = -INFINITY, slope = 0.0f;
                if (r < rows) {
                    const int s = slots ? slots[j] : j;
                    const float lse = wp.lse_in[((int64_t)b * p.S + s) * p.Hq + hq];
                    if (lse != -INFINITY) {
                        nlse = -lse * kLog2e;
                        own = cand0 + j;
                    } else none = true;
                    qp = p.pos ? p.pos[(int64_t)b * p.S + s] : cand0 + j;
                    slope = p.slopes ? p.slopes[hq] : 0.0f;
                }
                s_info[i] = make_float4(nlse, slope, __int_as_float(qp), __int_as_float(own));
                s_nlse[i] = nlse;
            }
            {   // a warp per head: 16-byte chunks of its rows
                constexpr int CPR = DP / 8, U = 4;
                for (int h = warp; h < p.H; h += WM)
                    for (int i0 = lane; i0 < rp * CPR; i0 += 32 * U) {
                        uint4 x[U];
#pragma unroll
                        for (int q = 0; q < U; ++q) {
                            const int i = i0 + q * 32, r = i / CPR, d = (i - r * CPR) * 8;
                            x[q] = make_uint4(0, 0, 0, 0);
                            if (r < rows && d < p.D) {
                                const int jr = r / p.G, j = j0 + jr, s = slots ? slots[j] : j;
                                x[q] = ld_nc16(static_cast<const T *>(p.q) + b * p.qsb + s * p.qss +
                                               (h * p.G + r - jr * p.G) * p.qsh + d);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < U; ++q) {
                            const int i = i0 + q * 32, r = i / CPR, d = (i - r * CPR) * 8;
                            if (r < rp) *reinterpret_cast<uint4 *>(sq + (size_t)(h * rp + r) * PITCH + d * 2) = x[q];
                        }
                    }
            }
            none = __syncthreads_or(none);
            // this lane's entries: rows g and g + 8 of the warp's 16
            int64_t off[2], off_next[2];
            auto look_up = [&](int t, int64_t (&o)[2]) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = it.keys.lo + t * WKT + warp * 16 + e * 8 + g;
                    o[e] = -1;
                    if (c < it.keys.hi) {
                        o[e] = entry_offset(p, table, c, 0);
                        if (o[e] < 0) attn_flag(p, b);
                    }
                }
            };
            uint4 k[2][NB][2];  // [buffer][32 columns][entry]
            auto load = [&](uint4 (&x)[NB][2], const int64_t (&o)[2], int h) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = i * 32 + q4 * 8;
                        x[i][e] = make_uint4(0, 0, 0, 0);
                        if (o[e] >= 0 && d < p.D) x[i][e] = ld_nc16(static_cast<const T *>(p.kc) + o[e] + (int64_t)h * p.D + d);
                    }
            };
            look_up(t0, off_next);
            load(k[0], off_next, 0);
            for (int t = t0; t < t1; ++t) {
                off[0] = off_next[0];
                off[1] = off_next[1];
                if (t + 1 < t1) look_up(t + 1, off_next);
                const int c0 = it.keys.lo + t * WKT + warp * 16;
                int kp[2];
                bool in[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = c0 + e * 8 + g;
                    in[e] = off[e] >= 0;
                    kp[e] = c;
                    if (in[e] && p.key_pos && c < cand0) kp[e] = p.key_pos[(int64_t)b * p.kps + c];
                    if (in[e] && c >= cand0 && p.pos) kp[e] = p.pos[(int64_t)b * p.S + (slots ? slots[c - cand0] : c - cand0)];
                    if (kp[e] < first) in[e] = false;
                }
                // candidates' own entries and the window mask by query
                const bool special = c0 + 16 > cand0 || p.window > 0;
                float acc[2] = {0.0f, 0.0f};
                const bool plain = !special && !none && p.score.cap == 0.0f && !p.score.bias;
                const float cf = p.score.scale * kLog2e;
                auto head = [&](const uint4 (&x)[NB][2], int h) {
                    const unsigned char *qr = sq + (size_t)(h * rp + g) * PITCH + q4 * 16;
                    const int q0 = h * rp + q4 * 2;
#pragma unroll 2
                    for (int r0 = 0; r0 < rp; r0 += 8) {
                        float y[4] = {0.f, 0.f, 0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(qr + r0 * PITCH + i * 64);
                            mma(y, x[i][0].x, x[i][1].x, x[i][0].y, x[i][1].y, v.x, v.y);
                            mma(z, x[i][0].z, x[i][1].z, x[i][0].w, x[i][1].w, v.z, v.w);
                        }
                        if (plain && r0 + 8 <= rows) {
                            const float2 nl = *reinterpret_cast<const float2 *>(s_nlse + q0 + r0);
                            acc[0] += ex2f(fmaf(y[0] + z[0], cf, nl.x)) + ex2f(fmaf(y[1] + z[1], cf, nl.y));
                            acc[1] += ex2f(fmaf(y[2] + z[2], cf, nl.x)) + ex2f(fmaf(y[3] + z[3], cf, nl.y));
                        } else {
#pragma unroll
                            for (int a = 0; a < 2; ++a) {
                                const float4 qi = s_info[q0 + r0 + a];
                                const int own = __float_as_int(qi.w), qp = __float_as_int(qi.z);
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int dist = pos_dist(qp, kp[e]);
                                    const float w = ex2f(fmaf(attn_score<false>(y[e * 2 + a] + z[e * 2 + a], p.score, qi.y, dist), kLog2e, qi.x));
                                    bool v = own >= 0;
                                    if (special) v = c0 + e * 8 + g <= own && (p.window == 0 || dist < p.window);
                                    acc[e] += v ? w : 0.0f;
                                }
                            }
                        }
                    }
                };
                for (int h = 0; h < p.H; h += 2) {
                    // two heads a turn, so that the buffers' indices are constants
                    if (h + 1 < p.H) load(k[1], off, h + 1);
                    else if (t + 1 < t1) load(k[1], off_next, 0);
                    head(k[0], h);
                    if (h + 1 < p.H) {
                        if (h + 2 < p.H) load(k[0], off, h + 2);
                        else if (t + 1 < t1) load(k[0], off_next, 0);
                        head(k[1], h + 1);
                    }
                }
                if (p.H & 1) {  // the next tile's first head is in the other buffer
#pragma unroll
                    for (int i = 0; i < NB; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) k[0][i][e] = k[1][i][e];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float a = in[e] ? acc[e] : 0.0f;
                    a += __shfl_xor_sync(kFull, a, 1);
                    a += __shfl_xor_sync(kFull, a, 2);
                    const int c = c0 + e * 8 + g;
                    if (in[e] && q4 == 0) wp.weight[b * wp.wstride + c] += a;
                    if (c < it.keys.hi && c >= cand0 && q4 == 1 && wp.key_pos_out && j0 == 0) {
                        const int j = c - cand0;
                        wp.key_pos_out[(int64_t)b * p.kps + c] = p.pos ? p.pos[(int64_t)b * p.S + (slots ? slots[j] : j)] : c;
                    }
                }
            }
        }
        u = it.u0 + it.ntiles;
        if (u >= uend) break;
        it = attn_next(p, it, 1, 1, WKT);
    }
}

template <int DP> cudaError_t launch_mma(const WeightsParams &p, int sms, cudaStream_t s) {
    // candidates a pass holds the queries of (K is read once per pass)
    const int row = WRow<DP>::kPitch + 20, heads = p.a.H * p.a.G;
    int per = kQueryBytes / (heads * row);
    while (per > 1 && (int64_t)p.a.H * ((per * p.a.G + 7) / 8 * 8) * row > kQueryBytes) --per;
    if (per < 1) per = 1;
    if (per > p.a.S) per = p.a.S;
    const int64_t smem = (int64_t)p.a.H * ((per * p.a.G + 7) / 8 * 8) * row;
    if (smem > 200 * 1024) return cudaErrorInvalidConfiguration;  // (launch_weights does not come here then)
    cudaError_t e = cudaFuncSetAttribute(weights_mma_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    weights_mma_kernel<DP><<<sms * (DP == 256 || smem > 100 * 1024 ? 1 : 2), WNT, (size_t)smem, s>>>(p, per);
    return cudaGetLastError();
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

cudaError_t launch_weights(const WeightsParams &p, int dtype, int sms, cudaStream_t s) {
    if (dtype != SPEC_DTYPE_BF16) return launch_t<float>(p, sms, s);
    WeightsParams t = p;
    t.a.box = attn_tc_box(p.a);
    const int per_pass = t.a.box ? weights_tc_per_pass(p.a) : 0;
    if (per_pass > 0) return launch_weights_tc(t, per_pass, sms, s);
    // one candidate's queries must fit: H * (G rounded up to 8) rows
    const int dp = p.a.D <= 64 ? 64 : p.a.D <= 128 ? 128 : 256;
    if ((int64_t)p.a.H * ((p.a.G + 7) / 8 * 8) * (dp * 2 + 36) > 200 * 1024) return launch_t<__nv_bfloat16>(p, sms, s);
    return dp == 64 ? launch_mma<64>(p, sms, s) : dp == 128 ? launch_mma<128>(p, sms, s) : launch_mma<256>(p, sms, s);
}

}  // namespace specv
