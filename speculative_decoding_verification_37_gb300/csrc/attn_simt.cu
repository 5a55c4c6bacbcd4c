// Attention over the paged cache on the CUDA cores, for float32 (the tensor cores
// would round its operands).
//
// Per (query, key): x = score(q . k), running maximum m and l = sum 2^(x - m),
// o = sum 2^(x - m) v, one pass over the keys (attention.cuh: the split over
// the grid and the join).  A block holds 16 or 32 queries, a quarter of them a
// warp, and 32 keys at a time in shared memory.  For the scores a lane has a key
// and reads its row once for all of the warp's queries, whose own elements are
// broadcast; for the values a lane has D/32 columns, and the weights are
// broadcast.  V is copied while the scores are taken, the next K during the rest.
//
// Bound by issue and shared-memory reads (a 16-byte read for each 16 FMA and one
// of K or V for the warp), not by HBM: 8 heads of 128, 64 x 5 queries on 2,048
// entries 719 us, 15 TFLOP/s; 16 single queries (4 a head) on up to 32,768,
// 780 us, 2.8 TB/s; 8 x 5 on up to 777, 2 heads of 72, 25 us in a graph.  Lanes
// of eight keys and a warp of four queries took 1,136 and 1,201 us, without the
// copies ahead 1,476 and 2,420; 64 queries a block 476 us where 32 take 409 (16
// requests of 13 x 4 queries a head on 2,048).
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
    float s[KT][RT + 4];   // softmax weights, a key's next to each other
    float o[RT][DP];
    float m[RT], l[RT];
    int kp[2][KT];         // two tiles' keys: position,
    int64_t koff[2][KT];   // element offset of the row; -1: none
    AttnRows<RT> rows;
    AttnPlan plan;
    int last;
};

// Blocks an SM holds: 32 rows of 128 columns want 168 registers a thread (64 x 5
// queries on 2,048 entries: 1,063 us in four blocks of 128, 719 in three, 867 in
// two), of 64 columns 128 (417 in four, 485 in three); 32 rows of 256 columns fill
// an SM's shared memory alone (a grid of two took turns on it: 16 requests of 5 x 4
// queries a head on 2,048 entries 595 us, of one 533; of 13 x 4 queries 1,141, 1,104).
constexpr int blocks_of(int DP, int R) { return DP == 256 ? (R == 1 ? 2 : 1) : R == 1 || DP == 64 ? 4 : 3; }

template <typename T, int DP, int R>
__global__ void __launch_bounds__(NT, blocks_of(DP, R)) attn_simt_kernel(AttnParams p) {
    constexpr int RW = 4 * R, RT = 4 * RW;       // rows of a warp, of the block
    constexpr int CW = DP < 128 ? 2 : 4, CB = DP / 32 / CW;  // columns of a lane: CB times CW neighbours
    extern __shared__ __align__(16) unsigned char raw[];
    SimtSmem<T, DP, RT> &sh = *reinterpret_cast<SimtSmem<T, DP, RT> *>(raw);
    static_assert(sizeof(T) == 4, "rows are copied as they are");
    const int tid = threadIdx.x, lane = tid & 31, row0 = (tid >> 5) * RW;  // this warp's rows
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
        float m[RW], l[RW], o[RW][CB * CW];  // m: the warp's, l: of this lane's keys
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < CB * CW; ++j) o[r][j] = 0.0f;
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
            float x[RW];  // this lane's key with the warp's rows
#pragma unroll
            for (int r = 0; r < RW; ++r) x[r] = 0.0f;
#pragma unroll 4
            for (int d = 0; d < DP; d += 4) {
                const float4 b = *reinterpret_cast<const float4 *>(&sh.k[lane][d]);
#pragma unroll
                for (int r = 0; r < RW; ++r) {
                    const float4 a = *reinterpret_cast<const float4 *>(&sh.q[row0 + r][d]);
                    x[r] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, x[r]))));
                }
            }
            if (t + 1 < t1) keep(t + 1);
            cp_async_wait_all();
            __syncthreads();
            if (t + 1 < t1) copy(t + 1, false);
            const bool there = s_koff[lane] >= 0;
            const int kp = s_kp[lane];
            bool hidden = false;  // from a row that there is
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                const int row = row0 + r;
                const bool is = sh.rows.out[row] >= 0;
                const int dist = pos_dist(sh.rows.qp[row], kp);
                if (is && there && attn_visible<RT>(p, it, sh.rows, row, c0 + lane, kp, dist)) {
                    x[r] = attn_score<true>(x[r], p.score, sh.rows.slope[row], dist);
                } else {
                    x[r] = -INFINITY;
                    hidden = hidden || is;
                }
                float mt = x[r];
#pragma unroll
                for (int q = 16; q > 0; q >>= 1) mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, q));
                // the reference m2 = max * log2(e), rounded; weights 2^(x*log2(e) - m2)
                const float m2 = fmaxf(m[r], mt * kLog2e), ref = m2 == -INFINITY ? 0.0f : m2;
                x[r] = x[r] == -INFINITY ? 0.0f : exp2f(fmaf(x[r], kLog2e, -ref));
                if (m2 > m[r]) {
                    const float corr = rel_weight(m[r], ref);
                    l[r] *= corr;
#pragma unroll
                    for (int j = 0; j < CB * CW; ++j) o[r][j] *= corr;
                }
                l[r] += x[r];
                m[r] = m2;
            }
#pragma unroll
            for (int r = 0; r < RW; r += 4)
                *reinterpret_cast<float4 *>(&sh.s[lane][row0 + r]) = make_float4(x[r], x[r + 1], x[r + 2], x[r + 3]);
            __syncwarp();
            const bool mask = __any_sync(kFull, hidden);  // a masked key's V may hold anything
#pragma unroll 4
            for (int k = 0; k < KT; ++k) {
                float w[RW], b[CB * CW];
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(&sh.s[k][row0 + r]);
                    w[r] = y.x, w[r + 1] = y.y, w[r + 2] = y.z, w[r + 3] = y.w;
                }
#pragma unroll
                for (int j = 0; j < CB; ++j) {
                    const float *from = &sh.v[k][(j * 32 + lane) * CW];
                    if (CW == 4) {
                        const float4 y = *reinterpret_cast<const float4 *>(from);
                        b[4 * j] = y.x, b[4 * j + 1] = y.y, b[4 * j + 2] = y.z, b[4 * j + 3] = y.w;
                    } else {
                        const float2 y = *reinterpret_cast<const float2 *>(from);
                        b[2 * j] = y.x, b[2 * j + 1] = y.y;
                    }
                }
                if (mask) {
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (w[r] != 0.0f) {
#pragma unroll
                            for (int j = 0; j < CB * CW; ++j) o[r][j] = fmaf(w[r], b[j], o[r][j]);
                        }
                } else {
#pragma unroll
                    for (int r = 0; r < RW; ++r)
#pragma unroll
                        for (int j = 0; j < CB * CW; ++j) o[r][j] = fmaf(w[r], b[j], o[r][j]);
                }
            }
            cp_async_wait_all();
            __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const int row = row0 + r;
#pragma unroll
            for (int j = 0; j < CB * CW; ++j) sh.o[row][(j / CW * 32 + lane) * CW + j % CW] = o[r][j];
#pragma unroll
            for (int q = 16; q > 0; q >>= 1) l[r] += __shfl_xor_sync(kFull, l[r], q);
            if (lane == 0) {
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
    constexpr int smem = (int)sizeof(SimtSmem<T, DP, 16 * R>);
    static_assert(blocks_of(DP, R) * (smem + 1024) <= 228 * 1024, "so many blocks' shared memory an SM has");
    cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<T, DP, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // (at most 8 / R blocks an SM: the workspace's partial results)
    const int grid = (sms < kAttnSmsMax ? sms : kAttnSmsMax) * blocks_of(DP, R);
    attn_simt_kernel<T, DP, R><<<grid, NT, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int DP> cudaError_t launch_r(const AttnParams &p, int sms, cudaStream_t s) {
    const int64_t rows = p.mode == 1 ? (int64_t)p.B * p.S * p.G : (int64_t)p.S * p.G;
    if (rows <= 16) return launch<T, DP, 1>(p, sms, s);
    return launch<T, DP, 2>(p, sms, s);
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
