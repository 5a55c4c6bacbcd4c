// Attention over the paged cache for bf16 and up to 64 rows per item
// (attention.cuh), on the warp-level tensor instructions.
//
// With few queries per cached head each K/V byte meets at most 64 rows, which
// the warp instructions keep up with: the kernel is bound by HBM.  One
// persistent block per SM streams its share of the line of tiles:
//   * four producer warps copy the keys' K and V rows (16-byte asynchronous
//     copies, completing on the stage's mbarrier) into a ring of stages, up to
//     about 170 KB ahead of the arithmetic, across item boundaries, so neither
//     the join of an item nor the next one's queries stop the stream.  Every
//     row has its own address, so pages may end anywhere in a tile, and a row
//     pitch of 16 bytes more than the data makes ldmatrix free of conflicts.
//     (One bulk copy per row instead: about 70 clocks each, 1.05 TB/s.);
//   * consumer warps split a tile's keys (32 each), from 33 rows on the rows,
//     and take turns at the tiles, so that several tiles are in work at once:
//     a warp's chain of dependent instructions per tile takes longer than the
//     tile's bytes.  Each warp
//     keeps its own running maximum, sum and output rows in registers (f32) and
//     never waits for another inside an item; at the item's end their results
//     are joined in shared memory in a fixed order.
// Measured (pages of 4): 64 requests of 5 queries on 2,048 entries of 8 heads of
// 128, 263 us, 2.1 TB/s; single queries on up to 32,768, 1,198 us, 3.7 TB/s
// (attn_tc.cu, where the pages allow it: 106 and 698).
// Scores and sums are f32; the softmax weights are rounded to bf16 for the
// product with V (at most 2^-8 of each weight, what the values carry
// themselves), their sum is taken before the rounding.
#include "attention.cuh"
#include "tma.cuh"

namespace specv {
namespace {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mbar_arrive(unsigned long long *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// 16 bytes, or zeros where `bytes` is 0
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// arrives on `bar` (one of its expected arrivals) once this thread's copies so far have landed
__device__ __forceinline__ void cp_async_arrive(unsigned long long *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 0xffff in each half that holds an infinity or NaN
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) { return __vcmpeq2(x & 0x7f807f80u, 0x7f807f80u); }

template <int DP, int MT, int WR, int WK, int NK, int NG, int ST> struct MmaCfg {
    static constexpr int kRows = 16 * MT * WR, kKeys = 16 * NK * WK, kWarps = WR * WK * NG, kNT = 32 * kWarps;
    static constexpr int kProducers = 4;
    // Producer warps take turns at the tiles, and so do the consumer groups.
    // The turns divide the ring: a stage then always has the same producer and
    // the same group, whose own order keeps every wait within one phase of its
    // barrier.  (With other counts one warp could be two fills ahead of
    // another at the same stage, where the phase bit says the opposite.)
    static constexpr int kTurns = ST % 4 == 0 ? 4 : ST % 3 == 0 ? 3 : 1;
    static_assert(ST % NG == 0 && ST % kTurns == 0, "turns divide the ring");
    // 8 consumer warps want more registers than 12 warps can have alike: the
    // producers hand over theirs (12 * 168 >= 4 * 56 + 8 * 224)
    static constexpr bool kSplitRegs = kWarps == 8;
    static constexpr int kPitch = DP * 2 + 16;  // bytes
};

template <int DP, int MT, int WR, int WK, int NK, int NG, int ST> struct MmaSmem {
    using C = MmaCfg<DP, MT, WR, WK, NK, NG, ST>;
    alignas(128) unsigned char kv[ST][2][C::kKeys * C::kPitch];
    alignas(16) unsigned char q[C::kRows * C::kPitch];
    alignas(16) float o[C::kRows][DP + 4];
    float m[WK * NG][C::kRows], l[WK * NG][C::kRows], tm[C::kRows], tl[C::kRows];
    int kp[ST][C::kKeys];          // positions, when key_pos is given
    unsigned valid[ST][C::kKeys / 32];  // bit per key
    AttnRows<C::kRows> rows;
    AttnPlan plan;
    alignas(8) unsigned long long full[ST], empty[ST];
    int last;
};

template <int DP, int MT, int WR, int WK, int NK, int NG, int ST>
__global__ void __launch_bounds__(32 * (WR * WK * NG + 4), 1) attn_mma_kernel(AttnParams p) {
    using C = MmaCfg<DP, MT, WR, WK, NK, NG, ST>;
    using T = __nv_bfloat16;
    constexpr int RT = C::kRows, KT = C::kKeys, NT = C::kNT, PITCH = C::kPitch;
    extern __shared__ __align__(128) unsigned char raw[];
    MmaSmem<DP, MT, WR, WK, NK, NG, ST> &sh = *reinterpret_cast<MmaSmem<DP, MT, WR, WK, NK, NG, ST> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = p.S * p.G;
    const int64_t nrows = p.mode == 1 ? (int64_t)p.B * per : per;
    const int rtiles = (int)((nrows + RT - 1) / RT);
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&sh.full[s], 32 + 1);
            mbar_init(&sh.empty[s], WR * WK);
        }
        fence_barrier_init();
    }
    // columns past D are never copied: zero once
    if (p.D < DP)
        for (int i = tid; i < (int)sizeof(sh.kv) / 16; i += NT + 32 * C::kProducers)
            reinterpret_cast<uint4 *>(sh.kv)[i] = make_uint4(0, 0, 0, 0);
    if (warp < C::kWarps) attn_plan<NT>(p, sh.plan, p.H * rtiles, KT);
    __syncthreads();
    const int64_t u0 = (int64_t)blockIdx.x * sh.plan.share;
    const int64_t uend = min(sh.plan.total, u0 + sh.plan.share);
    if (u0 >= uend) return;
    bool ok = true;  // after a wait has run out nothing waits any more; the call is flagged

    if (warp >= C::kWarps) {
        // ---------------- producers ----------------
        // They take turns at the tiles: a tile's fixed costs (the table's loads,
        // the waits) then overlap the other warps' copies.
        if (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        constexpr int CPR = DP / 8, KL = KT / 32;  // 16-byte chunks of a row; keys of a lane
        const int pw = warp - C::kWarps;
        if (pw >= C::kTurns) return;
        AttnItem it = attn_find<NT>(p, sh.plan, u0, p.H * rtiles, rtiles, KT);
        int n_issued = 0;
        int64_t u = u0;
        // V lies at a fixed distance from K, in the cache and among the candidates
        const int64_t v_cache = static_cast<const char *>(p.vc) - static_cast<const char *>(p.kc);
        const int64_t v_temp = static_cast<const char *>(p.tv) - static_cast<const char *>(p.tk);
        const int chunk = lane % CPR, sub = lane / CPR;
        const bool mine = chunk * 8 < p.D;
        while (true) {
            if (!it.keys.ok && u == it.u0 && it.h == 0 && it.rt == 0 && pw == 0 && lane == 0) attn_flag(p, it.b);
            const int t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
            const int *table = p.mode == 1 ? p.stable : p.table + (int64_t)it.b * p.max_blocks;
            for (int t = (int)(u - it.u0); t < t1; ++t, ++n_issued) {
                if (n_issued % C::kTurns != pw) continue;
                const int s = n_issued % ST;
                // the keys' K rows; bit 0: a candidate's, bit 1: no row (zeros are written)
                unsigned long long at[KL];
                unsigned v[KL];
                int kp[KL];
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    const int c = it.keys.lo + t * KT + j * 32 + lane;
                    at[j] = reinterpret_cast<unsigned long long>(p.kc) | 2ull;
                    kp[j] = 0;
                    if (c < it.keys.hi) {
                        if (p.tk && p.mode == 0 && c >= it.keys.len) {
                            at[j] = reinterpret_cast<unsigned long long>(
                                        static_cast<const T *>(p.tk) + (int64_t)it.b * p.tsb +
                                        ((int64_t)(c - it.keys.len) * p.H + it.h) * p.D) | 1ull;
                        } else {
                            const int64_t off = entry_offset(p, table, c, it.h);
                            if (off < 0) attn_flag(p, it.b);
                            else at[j] = reinterpret_cast<unsigned long long>(static_cast<const T *>(p.kc) + off);
                        }
                        if (p.key_pos) kp[j] = key_position(p, it, c);
                    }
                    v[j] = __ballot_sync(kFull, (at[j] & 2ull) == 0);
                }
                if (n_issued >= ST && ok) ok = attn_wait(&sh.empty[s], (unsigned)((n_issued / ST - 1) & 1));
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    if (p.key_pos) sh.kp[s][j * 32 + lane] = kp[j];
                    if (lane == 0) sh.valid[s][j] = v[j];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.full[s]);
                const uint32_t kd = smem_u32(sh.kv[s][0]) + (uint32_t)sub * PITCH + chunk * 16;
#pragma unroll
                for (int r = 0; r < KT; r += 32 / CPR) {
                    const unsigned long long a = __shfl_sync(kFull, at[r / 32], (r & 31) + sub);
                    if (mine) {
                        const char *k = reinterpret_cast<const char *>(a & ~3ull) + chunk * 16;
                        const int bytes = (a & 2ull) ? 0 : 16;
                        cp_async16(kd + r * PITCH, k, bytes);
                        cp_async16(kd + r * PITCH + KT * PITCH, k + ((a & 1ull) ? v_temp : v_cache), bytes);
                    }
                }
                cp_async_arrive(&sh.full[s]);
            }
            u = it.u0 + it.ntiles;
            if (u >= uend) break;
            it = attn_next(p, it, p.H * rtiles, rtiles, KT);
        }
        cp_async_wait_all();  // no copy may land after the block has gone
        if (!ok && lane == 0) atomicOr(p.status, SPEC_FLAG_TIMEOUT);
        return;
    }

    // ---------------- consumers ----------------
    if (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int grp = warp % NG, wk = warp / NG % WK, wr = warp / (NG * WK), kw = wk * NG + grp, g = lane >> 2, q4 = lane & 3;
    const int row0 = wr * MT * 16;
    const bool by_pos = p.window > 0 || p.first != nullptr;
    // ldmatrix lane addresses: Q and V take rows lane & 15, K rows by halves
    const uint32_t qa = smem_u32(sh.q) + (uint32_t)(row0 + (lane & 15)) * PITCH + (lane >> 4) * 16;
    const uint32_t ka = (uint32_t)(wk * 16 * NK + (lane & 7) + ((lane >> 4) << 3)) * PITCH + ((lane >> 3) & 1) * 16;
    const uint32_t va = (uint32_t)(wk * 16 * NK + (lane & 15)) * PITCH + (lane >> 4) * 16;
    int n_done = 0;
    int64_t u = u0;
    AttnItem it = attn_find<NT>(p, sh.plan, u0, p.H * rtiles, rtiles, KT);
    while (true) {
        attn_rows<RT, NT>(p, it, sh.rows, tid);
        sync_nt<NT>();
        for (int i = tid; i < RT * (DP / 8); i += NT) {
            const int r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (sh.rows.q[r] >= 0 && d < p.D) x = ld_nc16(static_cast<const T *>(p.q) + sh.rows.q[r] + d);
            *reinterpret_cast<uint4 *>(sh.q + r * PITCH + d * 2) = x;
        }
        sync_nt<NT>();
        float o[MT][DP / 8][4], m[MT][2], l[MT][2];
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            m[a][0] = m[a][1] = -INFINITY;
            l[a][0] = l[a][1] = 0.0f;
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) o[a][d][0] = o[a][d][1] = o[a][d][2] = o[a][d][3] = 0.0f;
        }
        const int t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
        for (int t = (int)(u - it.u0); t < t1; ++t, ++n_done) {
            if (n_done % NG != grp) continue;
            const int s = n_done % ST, c0 = it.keys.lo + t * KT + wk * 16 * NK;
            if (ok) ok = attn_wait(&sh.full[s], (unsigned)((n_done / ST) & 1));
            const uint32_t kb = smem_u32(sh.kv[s][0]) + ka, vb = smem_u32(sh.kv[s][1]) + va;
            float x[MT][2 * NK][4];
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int n = 0; n < 2 * NK; ++n) x[a][n][0] = x[a][n][1] = x[a][n][2] = x[a][n][3] = 0.0f;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                if (d * 16 < p.D) {
                    uint32_t b[NK][4];
#pragma unroll
                    for (int k = 0; k < NK; ++k) ldsm4(b[k], kb + k * 16 * PITCH + d * 32);
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        uint32_t f[4];
                        ldsm4(f, qa + a * 16 * PITCH + d * 32);
#pragma unroll
                        for (int k = 0; k < NK; ++k) {
                            mma16816(x[a][2 * k], f, b[k][0], b[k][1]);
                            mma16816(x[a][2 * k + 1], f, b[k][2], b[k][3]);
                        }
                    }
                }
            }
            const unsigned valid = NK == 2 ? sh.valid[s][wk] : (sh.valid[s][wk / 2] >> ((wk & 1) * 16)) & 0xffffu;
            const bool special = by_pos || valid != (NK == 1 ? 0xffffu : kFull) || (p.mode == 0 && c0 + 16 * NK > it.keys.len);
            bool hid = false;  // a masked key among this thread's
            if (special || p.score.bias) {
#pragma unroll
                for (int n = 0; n < 2 * NK; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = n * 8 + q4 * 2 + e, c = c0 + k;
                        const bool in = (valid >> k) & 1u;
                        const int kp = p.key_pos ? sh.kp[s][wk * 16 * NK + k] : in ? key_position(p, it, c) : 0;
#pragma unroll
                        for (int a = 0; a < MT; ++a)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int r = row0 + a * 16 + h * 8 + g;
                                const int dist = pos_dist(sh.rows.qp[r], kp);
                                float &y = x[a][n][h * 2 + e];
                                y = attn_score<false>(y, p.score, sh.rows.slope[r], dist);
                                if (special && !(in && attn_visible<RT>(p, it, sh.rows, r, c, kp, dist))) {
                                    y = -INFINITY;
                                    hid = true;
                                }
                            }
                    }
            } else {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int n = 0; n < 2 * NK; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[a][n][e] = attn_score<false>(x[a][n][e], p.score, 0.0f, 0);
            }
            // running maxima (log2 units), weights
            uint32_t pf[MT][NK][4];
            bool grew = false;
            float corr[MT][2];
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float mt = fmaxf(x[a][0][h * 2], x[a][0][h * 2 + 1]);
#pragma unroll
                    for (int n = 1; n < 2 * NK; ++n) mt = fmaxf(mt, fmaxf(x[a][n][h * 2], x[a][n][h * 2 + 1]));
                    mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 1));
                    mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 2));
                    const float mn = fmaxf(m[a][h], mt * kLog2e), ref = mn == -INFINITY ? 0.0f : mn;
                    corr[a][h] = rel_weight(m[a][h], ref);
                    grew = grew || mn > m[a][h];
                    m[a][h] = mn;
                    float sum = 0.0f;
#pragma unroll
                    for (int n = 0; n < 2 * NK; ++n) {
                        const float e0 = ex2f(fmaf(x[a][n][h * 2], kLog2e, -ref)), e1 = ex2f(fmaf(x[a][n][h * 2 + 1], kLog2e, -ref));
                        sum += e0 + e1;
                        pf[a][n / 2][(n & 1) * 2 + h] = pack_bf16(e0, e1);
                    }
                    l[a][h] = l[a][h] * corr[a][h] + sum;
                }
            if (__any_sync(kFull, grew)) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int d = 0; d < DP / 8; ++d) {
                        o[a][d][0] *= corr[a][0];
                        o[a][d][1] *= corr[a][0];
                        o[a][d][2] *= corr[a][1];
                        o[a][d][3] *= corr[a][1];
                    }
            }
            // a masked key's V may hold infinities or NaN, which a weight of 0
            // does not take out of a product: look for them where a key is masked
            bool dirty = false;
            if (__any_sync(kFull, hid)) {
                uint32_t found = 0;
#pragma unroll
                for (int k = 0; k < NK; ++k)
#pragma unroll 2
                    for (int d = 0; d < DP / 16; ++d) {
                        uint32_t b[4];
                        ldsm4t(b, vb + k * 16 * PITCH + d * 32);
                        found |= nonfinite2(b[0]) | nonfinite2(b[1]) | nonfinite2(b[2]) | nonfinite2(b[3]);
                    }
                dirty = __any_sync(kFull, found != 0u);
            }
            if (!dirty) {
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) {
                    if (d * 16 < p.D) {
#pragma unroll
                        for (int k = 0; k < NK; ++k) {
                            uint32_t b[4];
                            ldsm4t(b, vb + k * 16 * PITCH + d * 32);
#pragma unroll
                            for (int a = 0; a < MT; ++a) {
                                mma16816(o[a][2 * d], pf[a][k], b[0], b[1]);
                                mma16816(o[a][2 * d + 1], pf[a][k], b[2], b[3]);
                            }
                        }
                    }
                }
            } else {
                // the finite values as always; a visible key's non-finite value
                // makes its column NaN, found by a product of 0s and 1s
#pragma unroll
                for (int k = 0; k < NK; ++k)
#pragma unroll
                    for (int d = 0; d < DP / 16; ++d) {
                        uint32_t b[4], bad[4];
                        ldsm4t(b, vb + k * 16 * PITCH + d * 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            bad[i] = nonfinite2(b[i]);
                            b[i] &= ~bad[i];
                            bad[i] &= 0x3f803f80u;
                        }
#pragma unroll
                        for (int a = 0; a < MT; ++a) {
                            mma16816(o[a][2 * d], pf[a][k], b[0], b[1]);
                            mma16816(o[a][2 * d + 1], pf[a][k], b[2], b[3]);
                            uint32_t seen[4];
#pragma unroll
                            for (int n = 0; n < 2; ++n)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    seen[n * 2 + h] = (x[a][2 * k + n][h * 2] != -INFINITY ? 0x3f80u : 0u) |
                                                      (x[a][2 * k + n][h * 2 + 1] != -INFINITY ? 0x3f800000u : 0u);
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                float hit[4] = {0.f, 0.f, 0.f, 0.f};
                                mma16816(hit, seen, bad[2 * n], bad[2 * n + 1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (hit[e] > 0.0f) o[a][2 * d + n][e] = __int_as_float(0x7fffffff);
                            }
                        }
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[s]);
        }
        // join the warps of a row group
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float s = l[a][h];
                s += __shfl_xor_sync(kFull, s, 1);
                s += __shfl_xor_sync(kFull, s, 2);
                if (q4 == 0) {
                    sh.m[kw][row0 + a * 16 + h * 8 + g] = m[a][h];
                    sh.l[kw][row0 + a * 16 + h * 8 + g] = s;
                }
            }
        sync_nt<NT>();
        float f[MT][2];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = row0 + a * 16 + h * 8 + g;
                float mm = -INFINITY, ll = 0.0f;
#pragma unroll
                for (int w = 0; w < WK * NG; ++w) mm = fmaxf(mm, sh.m[w][r]);
#pragma unroll
                for (int w = 0; w < WK * NG; ++w) ll += sh.l[w][r] * rel_weight(sh.m[w][r], mm);
                f[a][h] = rel_weight(m[a][h], mm);
                if (kw == 0 && q4 == 0) {
                    sh.tm[r] = mm;
                    sh.tl[r] = ll;
                }
            }
        for (int w = 0; w < WK * NG; ++w) {
            if (kw == w) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int d = 0; d < DP / 8; ++d)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float2 *at = reinterpret_cast<float2 *>(&sh.o[row0 + a * 16 + h * 8 + g][d * 8 + q4 * 2]);
                            float2 v = make_float2(o[a][d][h * 2] * f[a][h], o[a][d][h * 2 + 1] * f[a][h]);
                            if (f[a][h] == 0.0f) v = make_float2(0.f, 0.f);  // this warp saw no key of the row
                            if (w > 0) {
                                const float2 b = *at;
                                v.x += b.x;
                                v.y += b.y;
                            }
                            *at = v;
                        }
            }
            sync_nt<NT>();
        }
        attn_finish<T, RT, NT>(p, sh.plan, it, sh.rows, &sh.o[0][0], DP + 4, sh.tm, sh.tl, &sh.last);
        u = it.u0 + it.ntiles;
        if (u >= uend) break;
        it = attn_next(p, it, p.H * rtiles, rtiles, KT);
    }
    if (!ok && lane == 0) atomicOr(p.status, SPEC_FLAG_TIMEOUT);
}

template <int DP, int MT, int WR, int WK, int NK, int NG, int ST> cudaError_t launch(const AttnParams &p, int sms, cudaStream_t s) {
    using C = MmaCfg<DP, MT, WR, WK, NK, NG, ST>;
    const int smem = (int)sizeof(MmaSmem<DP, MT, WR, WK, NK, NG, ST>);
    static_assert(sizeof(MmaSmem<DP, MT, WR, WK, NK, NG, ST>) <= 227 * 1024, "shared memory");
    static_assert(C::kRows <= kAttnSlotRows && C::kNT <= kAttnThreadsMax, "sizes");
    cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<DP, MT, WR, WK, NK, NG, ST>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = sms < kAttnSmsMax ? sms : kAttnSmsMax;
    attn_mma_kernel<DP, MT, WR, WK, NK, NG, ST><<<grid, C::kNT + 32 * C::kProducers, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Rows per block by the rows an item has: fewer row tiles re-read fewer keys.
cudaError_t launch_attn_mma(const AttnParams &p, int sms, cudaStream_t s) {
    const int64_t rows = p.mode == 1 ? (int64_t)p.B * p.S * p.G : (int64_t)p.S * p.G;
    const int size = rows <= 16 ? 0 : rows <= 32 ? 1 : 2;
    if (p.D <= 64)
        return size == 0 ? launch<64, 1, 1, 2, 2, 4, 8>(p, sms, s) : size == 1 ? launch<64, 2, 1, 2, 2, 4, 8>(p, sms, s)
                                                                               : launch<64, 2, 2, 2, 2, 2, 8>(p, sms, s);
    if (p.D <= 128)
        return size == 0 ? launch<128, 1, 1, 2, 2, 4, 4>(p, sms, s) : size == 1 ? launch<128, 2, 1, 2, 2, 4, 4>(p, sms, s)
                                                                                : launch<128, 2, 2, 2, 2, 2, 4>(p, sms, s);
    return size == 0 ? launch<256, 1, 1, 2, 1, 4, 4>(p, sms, s) : size == 1 ? launch<256, 1, 2, 2, 1, 2, 4>(p, sms, s)
                                                                            : launch<256, 1, 4, 2, 1, 1, 3>(p, sms, s);
}

}  // namespace specv
