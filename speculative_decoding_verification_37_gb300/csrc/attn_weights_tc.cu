// The attention weight cached entries accumulate (spec_attention_weights), for
// bf16 on the fifth-generation tensor cores.  Bound by HBM: K is read once.
//
// A tile is 128 entries of one request.  For each cached head K's rows are the
// 128 rows of an MMA and the head's queries its columns, so that one thread of
// an epilogue warp holds all scores of one entry: it adds exp(score - lse) up in
// a register over the heads, and nothing is exchanged but one number an entry
// between the two groups of epilogue warps, which take the heads in turn.  The
// queries of a request, all heads, lie in shared memory; TMA boxes bring K, 128
// KB ahead; four accumulators in TMEM keep the tensor cores, one epilogue group
// and the other apart.
//
// Measured (8 heads of 128, 4 queries each): 64 requests of 2,048 entries 62 us,
// 4.4 TB/s, of which 5 to 10 pass before the first product; 512 ragged ones of up
// to 4,096, 361 us, 6.1 TB/s; with capped and biased scores 394.  A query costs
// the epilogue an addition and an exponential an entry, a tanh two steps of the
// special-function unit more; leaving out the columns past the last query was
// worth 90 us, looking a tile's entries up a tile ahead 11.  K straight to
// registers on the warp instructions (attn_weights.cu), from the same pages of 16:
// 80 us for the first, 706 for the capped one.
#include "attn_tc.cuh"

namespace specv {
namespace {

constexpr int KT = 128, NT = 256;                 // entries of a tile, epilogue threads
constexpr int kColumns = 128;                     // queries of a cached head held at once
constexpr uint32_t kQueries = 80 * 1024;          // bytes: the queries of all heads held at once

template <int NH> struct WtSmem {                 // NH: 64-column halves of a head
    static constexpr uint32_t kTile = NH * KT * 128;
    static constexpr int kRing = 8 / NH, kInfo = (int)(kQueries / (NH * 128));
    alignas(1024) unsigned char k[kRing][kTile];
    alignas(1024) unsigned char q[kQueries];
    // the queries: -lse (log2 units; -inf: adds nothing), -slope (log2 units),
    // position, own entry (-1: adds nothing)
    alignas(16) float nlse[kInfo];
    alignas(16) float slope[kInfo];
    alignas(16) int qp[kInfo], own[kInfo];
    float part[2][KT];
    AttnPlan plan;
    alignas(8) unsigned long long full[kRing], empty[kRing], d_full[4], d_free[4], q_full;
    uint32_t tmem;
};

__device__ __forceinline__ bool bar_any(int id, int n, bool pred) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((int)pred), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

// A request's committed candidates (by a whole warp): none where it has no keys,
// -1 for bad data.
__device__ __forceinline__ int slots_of(const AttnParams &p, const AttnItem &it, int lane) {
    const int n = it.keys.ok ? p.n_slots[it.b] : 0;
    bool bad = !it.keys.ok;
    if (p.slots)
        for (int j = lane; j < n; j += 32) {
            const int s = p.slots[(int64_t)it.b * p.slots_stride + j];
            bad = bad || s < 0 || s >= p.S;
        }
    if (__any_sync(kFull, bad)) return -1;
    return it.keys.lo < it.keys.hi ? n : 0;
}

template <int NH, bool WH>
__global__ void __launch_bounds__(NT + 64, 1)
    weights_tc_kernel(const __grid_constant__ WeightsParams wp, const __grid_constant__ CUtensorMap map, int per_pass) {
    using Sm = WtSmem<NH>;
    using T = __nv_bfloat16;
    constexpr int NS = Sm::kRing;
    extern __shared__ unsigned char raw_[];
    Sm &sh = *reinterpret_cast<Sm *>(reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw_) + 1023) & ~uintptr_t(1023)));
    const AttnParams &p = wp.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.d_full[i], 1);
            mbar_init(&sh.d_free[i], NT / 2);
        }
        mbar_init(&sh.q_full, NT);
        fence_barrier_init();
    }
    if (warp < NT / 32) attn_plan<NT>(p, sh.plan, 1, KT);
    __syncthreads();
    int64_t u = (int64_t)blockIdx.x * sh.plan.share;
    const int64_t uend = min(sh.plan.total, u + sh.plan.share);
    if (u >= uend) return;
    if (warp == 0) tc_alloc(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    using Lay = TcLayout<NH, WH>;
    bool ok = true;  // after a wait has run out nothing waits any more; the call is flagged
    AttnItem it = attn_find<NT>(p, sh.plan, u, 1, 1, KT);

    if (warp == NT / 32) {
        // ---------------- TMA ----------------
        const int nbox = KT / p.box;
        const int zero_row = (int)(2 * p.nb * p.bs);  // past the map: zeros are written
        int n = 0;
        while (true) {
            const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0), slots = slots_of(p, it, lane);
            if (slots < 0 && u == it.u0 && lane == 0) attn_flag(p, it.b);
            if (slots >= 0 && u == it.u0) shared_positions(wp, it, lane, 32);
            const int *table = p.table + (int64_t)it.b * p.max_blocks;
            const KeyLine line = slots > 0 ? attn_line(p, it.keys) : KeyLine{0, 0};
            for (int j0 = 0; j0 < slots; j0 += per_pass)
                for (int t = t0; t < t1; ++t) {
                    int r = zero_row;
                    if (lane < nbox) {
                        const int k = t * KT + lane * p.box, c = line.lo + k;
                        if (k < line.entries) {
                            const int j = (int)fast_div((unsigned)c, p.bs_div), blk = __ldg(table + j);
                            if (blk < 0 || (int64_t)blk >= p.nb) attn_flag(p, it.b);
                            else r = blk * p.bs + (c - j * p.bs);
                        }
                    }
#pragma unroll 1
                    for (int h = 0; h < p.H; ++h, ++n) {
                        const int s = n % NS;
                        if (n >= NS && ok) ok = attn_wait(&sh.empty[s], (unsigned)((n / NS - 1) & 1));
                        if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], Sm::kTile);
                        __syncwarp();
                        if (lane < nbox) {
                            tc_copy_box<NH, WH>(smem_u32(sh.k[s]) + (uint32_t)(lane * p.box >> 3) * Lay::group, &map, r, h, &sh.full[s]);
                        }
                    }
                }
            u = it.u0 + it.ntiles;
            if (u >= uend) break;
            it = attn_next(p, it, 1, 1, KT);
        }
        // no copy may land after the block has gone
        for (int i = max(0, n - NS); i < n; ++i) ok = mbar_drain(&sh.full[i % NS], (unsigned)((i / NS) & 1)) && ok;
    } else if (warp == NT / 32 + 1) {
        // ---------------- MMA ----------------
        // Queries: a head's rows of one half of the columns, then of the other.
        const uint64_t dk = tc_desc(smem_u32(sh.k[0]), 16, Lay::group), dq = tc_desc(smem_u32(sh.q), 16, 1024);
        int n = 0, pass = 0;
        while (true) {
            const int nt = (int)(min(uend, it.u0 + it.ntiles) - u), slots = slots_of(p, it, lane);
            if (lane == 0)
                for (int j0 = 0; j0 < slots; j0 += per_pass, ++pass) {
                    const int rp = (min(per_pass, slots - j0) * p.G + 15) & ~15;
                    const uint32_t id = tc_idesc(rp, false), half = (uint32_t)rp * 128 / 16;
                    if (ok) ok = attn_wait(&sh.q_full, (unsigned)(pass & 1));
                    tc_fence_after();
                    for (int t = 0; t < nt; ++t)
#pragma unroll 1
                        for (int h = 0; h < p.H; ++h, ++n) {
                            const int s = n % NS, d = n & 3;
                            if (n >= 4 && ok) ok = attn_wait(&sh.d_free[d], (unsigned)(((n >> 2) - 1) & 1));
                            if (ok) ok = attn_wait(&sh.full[s], (unsigned)((n / NS) & 1));
                            tc_fence_after();
                            const uint64_t a = dk + (uint32_t)s * (Sm::kTile / 16), b = dq + (uint32_t)h * (NH * half);
#pragma unroll
                            for (int k = 0; k < NH * 4; ++k)
                                tc_mma_ss(tmem + d * kColumns, a + (k >> 2) * (Lay::half / 16) + (k & 3) * 32 / 16,
                                          b + (k >> 2) * half + (k & 3) * 32 / 16, id, k > 0);
                            tc_commit(&sh.empty[s]);
                            tc_commit(&sh.d_full[d]);
                        }
                }
            __syncwarp();
            u = it.u0 + it.ntiles;
            if (u >= uend) break;
            it = attn_next(p, it, 1, 1, KT);
        }
    } else {
        // ---------------- epilogue ----------------
        const int grp = warp >> 2, mrow = (warp & 3) * 32 + lane;  // TMEM lane = entry of the tile
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool cap = p.score.cap > 0.0f, bias = p.score.bias;
        const float cl = p.score.cap * kLog2e, cm = p.score.scale * (cap ? p.score.cap_arg : kLog2e);
        int n = 0, tiles = 0;
        while (true) {
            const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0), slots_n = slots_of(p, it, lane);
            const int b = it.b;
            const int *slots = p.slots ? p.slots + (int64_t)b * p.slots_stride : nullptr, *table = p.table + (int64_t)b * p.max_blocks;
            const int first = p.first ? p.first[b] : (int)0x80000000;
            const int cand0 = it.keys.len - slots_n;  // the candidates' first entry
            const KeyLine line = slots_n > 0 ? attn_line(p, it.keys) : KeyLine{0, 0};
            for (int j0 = 0; j0 < slots_n; j0 += per_pass) {
                // the queries (both groups are past the last pass's: its last tile's barrier)
                const int rows = min(per_pass, slots_n - j0) * p.G, rp = (rows + 15) & ~15;
                constexpr int CH = NH * 8, U = 8;  // 16-byte chunks of a query; loads in flight
#pragma unroll 1
                for (int i0 = tid; i0 < p.H * rp * CH; i0 += NT * U) {
                    uint4 x[U];
#pragma unroll
                    for (int q = 0; q < U; ++q) {
                        const int i = i0 + q * NT, row = i / CH, d = (i - row * CH) * 8, h = row / rp, r = row - h * rp;
                        x[q] = make_uint4(0, 0, 0, 0);
                        if (h < p.H && r < rows && d < p.D) {
                            const int jr = r / p.G, s = slots ? slots[j0 + jr] : j0 + jr;
                            x[q] = ld_nc16(static_cast<const T *>(p.q) + b * p.qsb + s * p.qss + (h * p.G + r - jr * p.G) * p.qsh + d);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < U; ++q) {
                        const int i = i0 + q * NT, row = i / CH, c = i - row * CH, h = row / rp, r = row - h * rp;
                        if (h >= p.H) continue;
                        *reinterpret_cast<uint4 *>(sh.q + ((uint32_t)(h * NH + (c >> 3)) * rp + r) * 128 + (((c & 7) ^ (r & 7)) << 4)) = x[q];
                    }
                }
                bool none = false;  // a query that adds nothing
                for (int i = tid; i < p.H * rp; i += NT) {
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
                        slope = p.slopes ? -p.slopes[hq] * kLog2e : 0.0f;
                    }
                    sh.nlse[i] = nlse;
                    sh.slope[i] = slope;
                    sh.qp[i] = qp;
                    sh.own[i] = own;
                }
                fence_async_shared();
                mbar_arrive(&sh.q_full);
                none = bar_any(1, NT, none);
                // this thread's entry of a tile: its block (-1: not there) and position
                int blk_next, kp_next;
                auto look_up = [&](int t) {
                    const int c = line.lo + t * KT + mrow;
                    blk_next = -1;
                    kp_next = c;
                    if (c < it.keys.lo || c >= it.keys.hi) return;
                    blk_next = __ldg(table + fast_div((unsigned)c, p.bs_div));
                    if (c >= cand0) {
                        if (p.pos) kp_next = p.pos[(int64_t)b * p.S + (slots ? slots[c - cand0] : c - cand0)];
                        if (grp == 0 && j0 == 0 && wp.key_pos_out) wp.key_pos_out[(int64_t)b * p.kps + c] = kp_next;
                    } else if (p.key_pos) {
                        kp_next = p.key_pos[(int64_t)b * p.kps + c];
                    }
                };
                look_up(t0);
                for (int t = t0; t < t1; ++t, ++tiles) {
                    const int c0 = line.lo + t * KT, c = c0 + mrow, kp = kp_next;
                    const bool in = blk_next >= 0 && (int64_t)blk_next < p.nb && kp >= first;
                    if (t + 1 < t1) look_up(t + 1);
                    // every query sees every entry
                    const bool all = c0 + KT <= cand0 && p.window == 0 && !none;
                    float acc[2] = {0.0f, 0.0f};
#pragma unroll 1
                    for (int h = 0; h < p.H; ++h, ++n) {
                        if ((n & 1) != grp) continue;
                        if (ok) ok = attn_wait(&sh.d_full[n & 3], (unsigned)((n >> 2) & 1));
                        tc_fence_after();
                        const uint32_t td = tl + (n & 3) * kColumns;
                        const int q0 = h * rp;
#pragma unroll 1
                        for (int r0 = 0; r0 < rows; r0 += 16) {
                            float x[16];  // becomes the score in log2 units
                            tc_ld16(x, td + r0);
                            tc_wait_ld();
#pragma unroll
                            for (int i8 = 0; i8 < 16; i8 += 8) {
                                if (r0 + i8 >= rows) break;
#pragma unroll
                                for (int i = i8; i < i8 + 8; i += 4) {
                                    const int q = q0 + r0 + i;
                                    const float4 l = *reinterpret_cast<const float4 *>(sh.nlse + q);
                                    float *y = x + i;
#pragma unroll
                                    for (int e = 0; e < 4; e += 2) {
                                        float2 v = __fmul2_rn(make_float2(y[e], y[e + 1]), make_float2(cm, cm));
                                        if (cap) {  // cap_score
                                            v = __fadd2_rn(make_float2(ex2f(v.x), ex2f(v.y)), make_float2(1.0f, 1.0f));
                                            v = __ffma2_rn(make_float2(rcpf(v.x), rcpf(v.y)), make_float2(-2.0f * cl, -2.0f * cl),
                                                           make_float2(cl, cl));
                                        }
                                        y[e] = v.x, y[e + 1] = v.y;
                                    }
                                    int dist[4];
                                    if (bias || !all) {
                                        const int4 qp = *reinterpret_cast<const int4 *>(sh.qp + q);
                                        dist[0] = pos_dist(qp.x, kp), dist[1] = pos_dist(qp.y, kp);
                                        dist[2] = pos_dist(qp.z, kp), dist[3] = pos_dist(qp.w, kp);
                                    }
                                    if (bias) {
                                        const float4 sl = *reinterpret_cast<const float4 *>(sh.slope + q);
                                        y[0] = fmaf(sl.x, (float)dist[0], y[0]);
                                        y[1] = fmaf(sl.y, (float)dist[1], y[1]);
                                        y[2] = fmaf(sl.z, (float)dist[2], y[2]);
                                        y[3] = fmaf(sl.w, (float)dist[3], y[3]);
                                    }
                                    y[0] = ex2f(y[0] + l.x), y[1] = ex2f(y[1] + l.y);
                                    y[2] = ex2f(y[2] + l.z), y[3] = ex2f(y[3] + l.w);
                                    if (!all || r0 + i + 4 > rows) {
                                        const int4 own = *reinterpret_cast<const int4 *>(sh.own + q);
                                        const int at[4] = {own.x, own.y, own.z, own.w};
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (c > at[e] || (p.window > 0 && !all && dist[e] >= p.window)) y[e] = 0.0f;
                                    }
                                    acc[0] += y[0] + y[1];
                                    acc[1] += y[2] + y[3];
                                  }
                            }
                        }
                        tc_fence_before();
                        mbar_arrive(&sh.d_free[n & 3]);
                    }
                    if (grp == 1) sh.part[tiles & 1][mrow] = acc[0] + acc[1];
                    bar_sync(1, NT);
                    if (grp == 0 && in) wp.weight[b * wp.wstride + c] += acc[0] + acc[1] + sh.part[tiles & 1][mrow];
                }
            }
            u = it.u0 + it.ntiles;
            if (u >= uend) break;
            it = attn_next(p, it, 1, 1, KT);
        }
    }
    if (!ok && lane == 0) atomicOr(p.status, SPEC_FLAG_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tc_dealloc(tmem);
}

template <int NH, bool WH> cudaError_t launch(const WeightsParams &p, int per_pass, int sms, cudaStream_t s) {
    constexpr int smem = (int)sizeof(WtSmem<NH>) + 1024;
    static_assert(smem <= 227 * 1024 && smem > 114 * 1024, "one block an SM: it takes all of TMEM");
    static_assert(WtSmem<NH>::kRing * NH == 8, "the ring");
    CUtensorMap map;
    if (!tc_cache_map(p.a, &map)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(weights_tc_kernel<NH, WH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    weights_tc_kernel<NH, WH><<<sms, NT + 64, smem, s>>>(p, map, per_pass);
    return cudaGetLastError();
}

}  // namespace

// Candidates whose queries a pass holds (K is read once per pass): at most
// kColumns rows of a cached head and kQueries bytes, rows in sixteens.
int weights_tc_per_pass(const AttnParams &p) {
    int rows = (int)(kQueries / ((uint32_t)p.H * (p.D <= 64 ? 128 : 256))) & ~15;
    if (rows > kColumns) rows = kColumns;
    return rows / p.G < p.S ? rows / p.G : p.S;
}

cudaError_t launch_weights_tc(const WeightsParams &p, int per_pass, int sms, cudaStream_t s) {
    if (p.a.D <= 64) return launch<1, true>(p, per_pass, sms, s);
    return p.a.D == 128 ? launch<2, true>(p, per_pass, sms, s) : launch<2, false>(p, per_pass, sms, s);
}

}  // namespace specv
