// Attention over the 8-bit paged cache for bf16 queries on the fifth-generation
// tensor cores (attention.cuh: score, split, join; kv8.cuh: the cache's numbers).
//
// The scheme is attn_tc.cu's: one persistent block per SM, tiles of 128 keys, the
// queries repeated C times down the 128 rows of the MMA, two groups of softmax warps
// that take turns at the tiles (one group above 64 rows).  What differs:
//   * K stays as it is.  S = Q K^T is a product of e4m3 operands: a query, scaled by
//     a power of two, is the sum of two e4m3 numbers (8 significant bits, as bf16
//     has; 2^-17 of the largest element is what the smallest may lose), both
//     products go into one accumulator.  A key's power of two multiplies its score;
//   * O = P V wants P's range: a weight of 2^-40 next to one of 1 is worth keeping
//     where there are many, and e4m3 ends at 2^-9.  So V's codes become bf16 (exactly:
//     the code's bits moved to their places, times 2^120), by the group that works at
//     the tile, a row a thread, before it looks at the scores.  Four codes need no
//     byte shuffles when the columns of O come as 0, 2, 1, 3; the end puts them back.
//     A key's power of two multiplies its weight before that is rounded to bf16;
//   * an entry whose V stands for NaN gives its NaN to the rows that give it weight,
//     by way of the power of two; its codes enter as finite numbers, so the rows
//     that it is hidden from see nothing.
// The copying warp also brings the tile's exponent bytes, four keys a lane.
//
#include "attention.cuh"
#include "attn_tc.cuh"
#include "kv8.cuh"
#include "tma.cuh"

namespace specv {
namespace {

constexpr int KT = 128;
constexpr uint32_t kTile = KT * 128;  // bytes: 128 keys x up to 128 codes; x 64 columns of bf16
constexpr int kInfo = 8;              // tiles whose notes are kept

__device__ __forceinline__ float2 pair(float a, float b) { return make_float2(a, b); }

// e4m3 x e4m3 -> f32, M = 128, both operands K-major
__host__ __device__ constexpr uint32_t tc_idesc8(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24); }
__device__ __forceinline__ void tc_mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Four codes as bf16, columns 0, 2 and 1, 3; `top` keeps the largest magnitudes
// (NaN's code comes out as 480, above any other).
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, __nv_bfloat162 &top) {
    const __nv_bfloat162 up = __halves2bfloat162(__ushort_as_bfloat16(0x7b80), __ushort_as_bfloat16(0x7b80));  // 2^120
    // sign to bit 15, exponent and mantissa to bits 10 .. 4: the value times 2^-120
    const uint32_t even = ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u);
    const uint32_t odd = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
    const __nv_bfloat162 a = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&even), up);
    const __nv_bfloat162 b = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&odd), up);
    top = __hmax2(top, __hmax2(__habs2(a), __habs2(b)));
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// How the softmax groups share the work: W = 0 one group, 1 tiles in turn.
template <int NH, int C, int W> struct Tc8Cfg {
    static constexpr int kRows = 128 / C;            // queries of an item
    static constexpr int kNT = W == 0 ? 128 : 256;   // softmax threads
    static constexpr int kThreads = kNT + 96;
    static constexpr int kCopies = W == 1 ? 2 * C : C;
    static constexpr uint32_t kV = NH * kTile;       // bytes of a V tile in bf16
    // the ring takes what the queries and V's buffers leave of 227 KB
    static constexpr int kRing = (NH == 1 ? 7 : 5) - (C == 1 ? 1 : 0);
};

template <int NH, int C, int W> struct Tc8Smem {
    using K = Tc8Cfg<NH, C, W>;
    alignas(1024) unsigned char kv[K::kRing][kTile];
    alignas(1024) unsigned char q[2][2][kTile];      // two items' queries, first and second parts
    alignas(1024) unsigned char v[2][K::kV];         // V in bf16; at an item's end the join's sums
    float m[K::kCopies][K::kRows], l[K::kCopies][K::kRows], tm[K::kRows], tl[K::kRows];
    float qs[2][K::kRows];                           // what the queries were divided by
    AttnRows<K::kRows> rows[2];
    alignas(16) int kp[2][KT];                       // a listed tile's keys: position,
    alignas(16) float kf[2][KT], vf[2][KT];          // a tile's powers of two
    unsigned sc[kInfo][2][KT / 4];                   // exponent bytes of a tile's K and V
    unsigned valid[2][4];                            // whether there is such a key
    unsigned bad[kInfo];                             // boxes of a tile with a bad block
    int low_max[2];                                  // the largest first visible position of an item's rows
    AttnPlan plan;
    alignas(8) unsigned long long full[K::kRing], empty[K::kRing], s_full[2], p_full[2], pv_done[2], q_full[2], q_free[2];
    uint32_t tmem;
    int last;
};

// a barrier of n threads under an id of its own that joins a predicate
__device__ __forceinline__ bool bar_or(int id, int n, bool pred) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((int)pred), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

template <int NH, int C, int W>
__global__ void __launch_bounds__(Tc8Cfg<NH, C, W>::kThreads, 1)
    attn8_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap cache_map) {
    using K = Tc8Cfg<NH, C, W>;
    using T = __nv_bfloat16;
    constexpr int RT = K::kRows, NT = K::kNT, NS = K::kRing, NC = KT / C;
    constexpr int CH = NC < 64 ? 32 : 64;  // scores a thread holds at once
    extern __shared__ unsigned char raw_[];
    Tc8Smem<NH, C, W> &sh = *reinterpret_cast<Tc8Smem<NH, C, W> *>(
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw_) + 1023) & ~uintptr_t(1023)));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = p.S * p.G;
    const int64_t nrows = p.mode == 1 ? (int64_t)p.B * per : per;
    const int rtiles = (int)((nrows + RT - 1) / RT), items = p.H * rtiles;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 128);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.q_full[i], 32);
            mbar_init(&sh.q_free[i], NT);
        }
        fence_barrier_init();
    }
    if (W != 1) {  // (the marks of the shared pass have been read)
        pdl_wait_primary();
        attn_begin(p);
    }
    if (warp < NT / 32) attn_plan<NT>(p, sh.plan, items, KT);
    __syncthreads();
    if (W != 1) pdl_launch_dependents();
    int64_t u = (int64_t)blockIdx.x * sh.plan.share;
    const int64_t uend = min(sh.plan.total, u + sh.plan.share);
    if (u >= uend) return;
    if (warp == 0) tc_alloc(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // TMEM columns: two score tiles (P lies over the first half of each), then
    // one or two accumulators
    constexpr uint32_t kS = 0, kO = 256;
    bool ok = true;  // after a wait has run out nothing waits any more; the call is flagged
    AttnItem it = attn_find<NT>(p, sh.plan, u, items, rtiles, KT);

    if (warp == NT / 32) {
        // ---------------- TMA ----------------
        const int nbox = KT / p.box;
        const int zero_row = (int)(2 * p.nb * p.bs);  // past the map: zeros are written
        const int v_row = (int)(p.nb * p.bs);
        int n = 0, tiles = 0;
        while (true) {
            if (!it.keys.ok && u == it.u0 && it.h == 0 && it.rt == 0 && lane == 0) attn_flag(p, it.b);
            const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
            const int *table = p.mode == 1 ? p.stable : p.table + (int64_t)it.b * p.max_blocks;
            const KeyLine line = it.keys.ok ? attn_line(p, it.keys) : KeyLine{0, 0};
            int row_k = 0, row_v = 0;      // this lane's box: row of the cache
            unsigned ks = 0u, vs = 0u, ks_before = 0u, vs_before = 0u;
            // a lane looks up 4 keys (a page has a multiple of 8), and takes its box's
            // row from the lane that has the first of them
            auto look_up = [&](int t) {
                int r = zero_row;
                bool bad = false;
                const int k = t * KT + lane * 4, c = line.lo + k;
                ks = vs = 0u;
                if (k < line.entries && c < it.keys.hi) {
                    const int j = (int)fast_div((unsigned)c, p.bs_div), at = c - j * p.bs, blk = __ldg(table + j);
                    bad = blk < 0 || (int64_t)blk >= p.nb;
                    if (!bad) {
                        r = blk * p.bs + at;
                        const int64_t s = ((int64_t)blk * p.H + it.h) * p.bs + at;
                        ks = __ldg(reinterpret_cast<const unsigned *>(p.ks + s));
                        vs = __ldg(reinterpret_cast<const unsigned *>(p.vs + s));
                    }
                }
                if (bad) attn_flag(p, it.b);
                const int from = lane < nbox ? lane * p.box >> 2 : 0;
                const bool box_bad = __shfl_sync(kFull, (int)bad, from) != 0;
                r = __shfl_sync(kFull, r, from);
                const unsigned b = __ballot_sync(kFull, box_bad && lane < nbox);
                if (lane == 0) sh.bad[tiles % kInfo] = b;
                ++tiles;
                return r;
            };
            auto copy = [&](int r, bool is_v) {
                const int s = n % NS;
                if (n >= NS && ok) ok = attn_wait(&sh.empty[s], (unsigned)((n / NS - 1) & 1));
                __syncwarp();  // (the notes of all lanes, before the arrival)
                if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], kTile);
                __syncwarp();
                if (lane < nbox) {
                    const uint32_t dst = smem_u32(sh.kv[s]) + (uint32_t)(lane * p.box) * 128u;
                    tma3(dst, &cache_map, 0, it.h, is_v && r != zero_row ? r + v_row : r, &sh.full[s]);
                }
                ++n;
            };
            // the order of use: K0 K1 V0 K2 V1 ...
#pragma unroll 1
            for (int t = t0; t < t1 + 1; ++t) {
                row_v = row_k;
                ks_before = ks, vs_before = vs;
                if (t < t1) {
                    row_k = look_up(t);
                    copy(row_k, false);
                }
                if (t > t0) {  // (the bytes have had the time of a tile to arrive)
                    const int i = (tiles - (t < t1 ? 2 : 1)) % kInfo;
                    sh.sc[i][0][lane] = ks_before;
                    sh.sc[i][1][lane] = vs_before;
                    copy(row_v, true);
                }
            }
            u = it.u0 + it.ntiles;
            if (u >= uend) break;
            it = attn_next(p, it, items, rtiles, KT);
        }
        // no copy may land after the block has gone
        for (int i = max(0, n - NS); i < n; ++i) ok = mbar_drain(&sh.full[i % NS], (unsigned)((i / NS) & 1)) && ok;
    } else if (warp == NT / 32 + 1) {
        // ---------------- MMA ----------------
        if (lane == 0) {
            // Operands in atoms of 8 rows x 128 bytes, the next 8 rows 1,024 bytes on.
            // 32 columns of K and Q are 32 bytes; V's columns are its N, contiguous
            // (lbo: the next 64 columns, sbo: the next 8 keys).
            constexpr uint32_t id_s = tc_idesc8(KT), id_o = tc_idesc(NH * 64, true);
            const uint64_t dq = tc_desc(smem_u32(sh.q[0][0]), 16, 1024), dk = tc_desc(smem_u32(sh.kv[0]), 16, 1024),
                           dv = tc_desc(smem_u32(sh.v[0]), kTile, 1024);
            int n = 0, j = 0, item = 0;
            while (true) {
                const int nt = (int)(min(uend, it.u0 + it.ntiles) - u);
                if (ok) ok = attn_wait(&sh.q_full[item & 1], (unsigned)((item >> 1) & 1));
                tc_fence_after();
                // S0 S1, P0 V0, S2, P1 V1, S3 ...
                const int j0 = j;
#pragma unroll 1
                for (int i = 0; i < nt + 2; ++i) {
                    if (i >= 2) {
                        const int b = j & 1;  // score tile, buffer of V
                        if (ok) ok = attn_wait(&sh.p_full[b], (unsigned)((j >> 1) & 1));
                        tc_fence_after();
                        const uint64_t at = dv + (uint32_t)b * (K::kV / 16);
                        const uint32_t o = tmem + kO + (W == 0 ? 0 : b) * 128, pt = tmem + kS + b * 128;
                        const bool first = W == 0 ? i == 2 : i < 4;
#pragma unroll
                        for (int k = 0; k < KT / 16; ++k) tc_mma_ts(o, pt + k * 8, at + k * (2048 / 16), id_o, !(first && k == 0));
                        tc_commit(&sh.pv_done[W == 0 ? 0 : b]);
                        ++n;
                        ++j;
                    }
                    if (i < nt) {
                        const int d = (j0 + i) & 1;
                        if (ok) ok = attn_wait(&sh.full[n % NS], (unsigned)((n / NS) & 1));
                        tc_fence_after();
                        const uint64_t a = dq + (uint32_t)(item & 1) * (2 * kTile / 16), b = dk + (uint32_t)(n % NS) * (kTile / 16);
#pragma unroll
                        for (int k = 0; k < NH * 4; ++k)  // first parts, second parts
                            tc_mma8(tmem + kS + d * 128, a + (k / (NH * 2)) * (kTile / 16) + (k % (NH * 2)) * (32 / 16),
                                    b + (k % (NH * 2)) * (32 / 16), id_s, k > 0);
                        tc_commit(&sh.empty[n % NS]);
                        tc_commit(&sh.s_full[d]);
                        ++n;
                    }
                }
                ++item;
                u = it.u0 + it.ntiles;
                if (u >= uend) break;
                it = attn_next(p, it, items, rtiles, KT);
            }
        }
        __syncwarp();
    } else if (warp == NT / 32 + 2) {
        // ---------------- queries ----------------
        // The next item's rows and queries, while this one's keys go by: a group of
        // lanes a row, 8 elements a lane.
        const bool by_pos = p.window > 0 || p.first != nullptr;
        const uint32_t neg = p.score.scale < 0.0f ? 0x80008000u : 0u;  // a negative scale: the queries are negated
        for (int item = 0;; ++item) {
            const int qb = item & 1;
            // the buffer's last item, and its rows, are done with
            if (item >= 2 && ok) ok = attn_wait(&sh.q_free[qb], (unsigned)((item / 2 - 1) & 1));
            AttnRows<RT> &w = sh.rows[qb];
            attn_rows<RT, 32>(p, it, w, lane);
            __syncwarp();
            int low = (int)0x80000000;
            if (by_pos)
                for (int i = lane; i < RT; i += 32)
                    if (w.out[i] >= 0) low = max(low, max(w.first[i], p.window > 0 ? w.qp[i] - p.window + 1 : (int)0x80000000));
            low = __reduce_max_sync(kFull, low);
            if (lane == 0) sh.low_max[qb] = low;
            constexpr int LR = NH * 8, RW = 32 / LR, U = 8;  // lanes of a row; rows a load; loads in flight
            const int d = (lane % LR) * 8;
#pragma unroll 1
            for (int r0 = 0; r0 < RT; r0 += RW * U) {
                uint4 v[U];
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const int r = r0 + q * RW + lane / LR;
                    v[q] = make_uint4(0, 0, 0, 0);
                    if (w.q[r] >= 0 && d < p.D) v[q] = ld_nc16(static_cast<const T *>(p.q) + w.q[r] + d);
                }
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const int r = r0 + q * RW + lane / LR;
                    v[q].x ^= neg, v[q].y ^= neg, v[q].z ^= neg, v[q].w ^= neg;
                    float x[8], top = 0.0f;
                    unpack<T>(v[q], x);
                    if (nonfinite2(v[q].x) | nonfinite2(v[q].y) | nonfinite2(v[q].z) | nonfinite2(v[q].w)) top = INFINITY;
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
                    for (int i = LR / 2; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
                    const unsigned s = kv8_scale(top);
                    const float f = s == 255u ? 0.0f : kv8_inverse(s);
                    if (lane % LR == 0) sh.qs[qb][r] = kv8_power(s);
                    uint32_t a[2], b[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        a[i] = kv8_code2(x[4 * i] * f, x[4 * i + 1] * f) | kv8_code2(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16;
                        const float4 y = kv8_value4(a[i]);
                        b[i] = kv8_code2(x[4 * i] * f - y.x, x[4 * i + 1] * f - y.y) |
                               kv8_code2(x[4 * i + 2] * f - y.z, x[4 * i + 3] * f - y.w) << 16;
                    }
#pragma unroll
                    for (int k = 0; k < C; ++k) {
                        const int mr = r + k * RT;
                        const uint32_t at = mr * 128 + (((d >> 4) ^ (mr & 7)) << 4) + (d & 8);
                        *reinterpret_cast<uint2 *>(sh.q[qb][0] + at) = make_uint2(a[0], a[1]);
                        *reinterpret_cast<uint2 *>(sh.q[qb][1] + at) = make_uint2(b[0], b[1]);
                    }
                }
            }
            fence_async_shared();
            mbar_arrive(&sh.q_full[qb]);
            u = it.u0 + it.ntiles;
            if (u >= uend) break;
            it = attn_next(p, it, items, rtiles, KT);
        }
        __syncwarp();
    } else {
        // ---------------- softmax ----------------
        const int wq = warp & 3, grp = warp >> 2;                 // TMEM lanes 32 wq .. + 31
        const int mrow = wq * 32 + lane;                          // row of the MMA; key of a tile
        const int copy = C == 1 ? 0 : wq / (4 / C);
        const int row = mrow % RT;                                // query of the item
        const int cb = copy * NC;                                 // first key of the copy in a tile
        const int acc = W == 0 ? 0 : grp;                         // accumulator
        const int bar = W == 1 ? 2 + grp : 1, nbar = 128;         // the threads that share a tile
        const uint32_t tl = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t to = tl + kO + acc * 128;
        const bool by_pos = p.window > 0 || p.first != nullptr;
        float *so = reinterpret_cast<float *>(sh.v[0]);           // the join's sums, once all products have ended
        constexpr int LD = NH * 64 + 4;
        static_assert(W != 1 || RT * LD * 4 <= 2 * (int)K::kV, "they fit V's buffers");
        int item = 0, j = 0, nring = 0;
        while (true) {
            const int qb = item & 1;
            if (ok) ok = attn_wait(&sh.q_full[qb], (unsigned)((item >> 1) & 1));
            const AttnRows<RT> &w = sh.rows[qb];
            const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0), nt = t1 - t0;
            const int qp = w.qp[row], cand = w.cand[row];
            const int low = max(w.first[row], p.window > 0 ? qp - p.window + 1 : (int)0x80000000);
            const float slope = w.slope[row], scale = fabsf(p.score.scale) * sh.qs[qb][row];
            const KeyLine line = it.keys.ok ? attn_line(p, it.keys) : KeyLine{0, 0};
            float m = -INFINITY, l = 0.0f;  // reference (log2 units), sum
            // position of key `mrow` of tile t, when key_pos is given: read a tile ahead
            auto key_pos_of = [&](int t) {
                const int k = t * KT + mrow, c = line.lo + k;
                return k < line.entries && c < it.keys.len ? __ldg(p.key_pos + (int64_t)it.b * p.kps + c) : 0;
            };
            const int step = W == 1 ? 2 : 1, first = W == 1 && (j & 1) != grp ? t0 + 1 : t0;
            int kp_next = p.key_pos && first < t1 ? key_pos_of(first) : 0;
            const int j0 = j;
            for (int t = first; t < t1; t += step) {
                const int tt = t - t0, jj = j0 + tt;               // tiles of the block so far
                const int sb = W == 0 ? jj & 1 : grp;              // score tile, buffers
                const int kp_mine = kp_next;
                if (p.key_pos && t + step < t1) kp_next = key_pos_of(t + step);
                // V's buffer is free once the product that read it has ended (W = 0: seen
                // with the tile before)
                if (W == 1 && t > first) {
                    if (ok) ok = attn_wait(&sh.pv_done[grp], (unsigned)(((jj - 2) >> 1) & 1));
                    tc_fence_after();
                }
                // V of this tile: its place in the ring by the order of the copies
                const int nv = nring + (tt + 1 < nt ? 2 * tt + 2 : 2 * tt + 1);
                if (ok) ok = attn_wait(&sh.full[nv % NS], (unsigned)((nv / NS) & 1));
                {
                    const unsigned char *from = sh.kv[nv % NS] + mrow * 128;
                    unsigned char *dst = sh.v[sb] + mrow * 128;
                    __nv_bfloat162 top = __halves2bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
#pragma unroll
                    for (int i = 0; i < NH * 4; ++i) {  // 16 columns
                        const uint4 y = *reinterpret_cast<const uint4 *>(from + ((i ^ (mrow & 7)) << 4));
                        const uint2 a = codes_to_bf16(y.x, top), b = codes_to_bf16(y.y, top), c = codes_to_bf16(y.z, top),
                                    d = codes_to_bf16(y.w, top);
                        unsigned char *half = dst + (i >> 2) * kTile;
                        const int at = (i & 3) * 2;
                        *reinterpret_cast<uint4 *>(half + ((at ^ (mrow & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
                        *reinterpret_cast<uint4 *>(half + (((at + 1) ^ (mrow & 7)) << 4)) = make_uint4(c.x, c.y, d.x, d.y);
                    }
                    fence_async_shared();
                    const unsigned char *sc = reinterpret_cast<const unsigned char *>(sh.sc[jj % kInfo][0]);
                    const bool nan = __bfloat162float(__hmax(__low2bfloat16(top), __high2bfloat16(top))) > 448.0f;
                    const unsigned char vs = nan ? 255 : sc[KT + mrow];
                    sh.kf[sb][mrow] = kv8_power(sc[mrow]);
                    sh.vf[sb][mrow] = kv8_power(vs);
                }
                const bool nanv = bar_or(bar, nbar, sh.vf[sb][mrow] != sh.vf[sb][mrow]);
                if (mrow == 0) mbar_arrive(&sh.empty[nv % NS]);
                if (ok) ok = attn_wait(&sh.s_full[sb], (unsigned)((jj >> 1) & 1));
                tc_fence_after();
                const uint32_t ts = tl + kS + sb * 128 + cb;       // this thread's scores
                const float *kf = sh.kf[sb] + cb, *vf = sh.vf[sb] + cb;
                const int k0 = t * KT, c0 = line.lo + k0;
                // whether the tile may mask a key: the line's ends, candidates, a bad
                // block, the window's and the document's first tile
                const bool special = !it.keys.ok || c0 < it.keys.lo || c0 + KT > it.keys.len || k0 + KT > line.entries ||
                                     sh.bad[jj % kInfo] != 0u || (by_pos && (p.key_pos || c0 < sh.low_max[qb]));
                const bool listed = special || (p.key_pos && p.score.bias);
                const int q0 = it.keys.len - c0;                   // the tile's first candidate, as an index into the tile
                if (listed) {
                    const int k = k0 + mrow, c = c0 + mrow;
                    bool in = false;
                    int kp = 0;
                    if (it.keys.ok && k < line.entries && c >= it.keys.lo && c < it.keys.hi &&
                        !((sh.bad[jj % kInfo] >> (mrow / p.box)) & 1u)) {
                        in = true;
                        kp = c < it.keys.len ? (p.key_pos ? kp_mine : c) : key_position(p, it, c);
                    }
                    const unsigned b = __ballot_sync(kFull, in);
                    if (lane == 0) sh.valid[sb][wq] = b;
                    sh.kp[sb][mrow] = kp;
                    bar_sync(bar, nbar);
                }
                const bool plain = !listed && p.score.cap == 0.0f && !p.score.bias;
                float x[CH];
                auto load = [&](int i) {  // scores i .. i + CH - 1, but for the query's factor
                    tc_ldx<CH>(x, ts + i);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < CH; e += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(kf + i + e);
                        const float2 a = __fmul2_rn(pair(x[e], x[e + 1]), pair(f.x, f.y)), b = __fmul2_rn(pair(x[e + 2], x[e + 3]), pair(f.z, f.w));
                        x[e] = a.x, x[e + 1] = a.y, x[e + 2] = b.x, x[e + 3] = b.y;
                    }
                };
                float cf = scale * kLog2e, mt = -INFINITY;
                if (plain) {
#pragma unroll
                    for (int i = 0; i < NC; i += CH) {
                        load(i);
                        mt = fmaxf(mt, max_of<CH>(x));
                    }
                } else {
                    // scores in natural units, 32 at a time, and back into TMEM
                    cf = kLog2e;
#pragma unroll 1
                    for (int i = 0; i < NC; i += 32) {
                        float y[32];
                        tc_ldx<32>(y, ts + i);
                        tc_wait_ld();
                        const bool capped = p.score.cap > 0.0f;
                        const float s = capped ? scale * p.score.cap_arg : scale, c2 = -2.0f * p.score.cap;
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(kf + i + e);
                            // (the key's factor first: with the query's it is the score's size)
                            float2 a = __fmul2_rn(pair(y[e], y[e + 1]), pair(f.x, f.y)), b = __fmul2_rn(pair(y[e + 2], y[e + 3]), pair(f.z, f.w));
                            a = __fmul2_rn(a, pair(s, s));
                            b = __fmul2_rn(b, pair(s, s));
                            y[e] = a.x, y[e + 1] = a.y, y[e + 2] = b.x, y[e + 3] = b.y;
                        }
                        if (capped) {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {  // cap_score
                                const float2 v = __fadd2_rn(pair(ex2f(y[e]), ex2f(y[e + 1])), pair(1.0f, 1.0f));
                                const float2 z = __ffma2_rn(pair(rcpf(v.x), rcpf(v.y)), pair(c2, c2), pair(p.score.cap, p.score.cap));
                                y[e] = z.x, y[e + 1] = z.y;
                            }
                        }
                        const int *kp = sh.kp[sb] + cb + i;
                        if (p.score.bias) {
                            const float2 ns = pair(-slope, -slope);
                            if (listed) {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 v = __ffma2_rn(ns, pair((float)pos_dist(qp, kp[e]), (float)pos_dist(qp, kp[e + 1])), pair(y[e], y[e + 1]));
                                    y[e] = v.x, y[e + 1] = v.y;
                                }
                            } else {
                                const float d0 = (float)(qp - (c0 + cb + i));
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 v = __ffma2_rn(ns, __fadd2_rn(pair(d0, d0), pair((float)-e, (float)(-e - 1))), pair(y[e], y[e + 1]));
                                    y[e] = v.x, y[e + 1] = v.y;
                                }
                            }
                        }
                        if (special) {
                            // bit e: key e of the chunk is seen by this row
                            unsigned seen = sh.valid[sb][(cb + i) / 32];
                            const int q = cb + i - q0;        // the chunk's first key as a candidate
                            if (p.mode == 0 && q > -32) {
                                unsigned mine = 0u;           // candidates q .. q + 31
                                if (p.mask) {
                                    const uint32_t *mw = p.mask + ((int64_t)it.b * p.S + cand) * p.W;
                                    const int w0 = q >> 5;    // (floor)
                                    const uint32_t a = w0 >= 0 && w0 < p.W ? mw[w0] : 0u, b = w0 + 1 < p.W ? mw[w0 + 1] : 0u;
                                    mine = __funnelshift_r(a, b, q & 31);
                                } else if (cand >= q) {
                                    mine = cand - q >= 31 ? kFull : (2u << (cand - q)) - 1u;
                                }
                                // keys before the first candidate are entries
                                if (q < 0) mine |= (1u << -q) - 1u;
                                seen &= mine;
                            }
                            if (by_pos) {
                                unsigned near = 0u;
#pragma unroll
                                for (int e = 0; e < 32; ++e) near |= (unsigned)(kp[e] >= low) << e;
                                seen &= near;
                            }
#pragma unroll
                            for (int e = 0; e < 32; ++e) y[e] = (seen >> e) & 1u ? y[e] : -INFINITY;
                        }
                        mt = fmaxf(mt, max_of<32>(y));
                        uint32_t z[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) z[e] = __float_as_uint(y[e]);
                        tc_st32(ts + i, z);
                    }
                    tc_wait_st();
                }
                mt *= cf;
                // a new reference when the maximum has grown past 2^8 of the old one
                const bool grew = mt > m + 8.0f || (m == -INFINITY && mt > -INFINITY);
                float corr = 1.0f;
                if (grew) {
                    corr = rel_weight(m, mt);
                    m = mt;
                    l *= corr;
                }
                if (W == 0 && t > first) {
                    // every product's end is seen before the next is let go: the
                    // barrier's phase bit tells only neighbours apart
                    if (ok) ok = attn_wait(&sh.pv_done[0], (unsigned)((jj - 1) & 1));
                    tc_fence_after();
                }
                if (__any_sync(kFull, grew) && t > first) {
#pragma unroll 1
                    for (int d = 0; d < NH * 64; d += 32) {
                        float o[32];
                        uint32_t y[32];
                        tc_ld32(o, to + d);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(o[i] * corr);
                        tc_st32(to + d, y);
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                const uint32_t pt = tl + kS + sb * 128 + cb / 2;
                const float2 cf2 = pair(cf, cf), nref = pair(-ref, -ref);
                float2 sum0 = pair(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
                for (int i = 0; i < NC; i += CH) {
                    if (!plain) {
                        tc_ldx<CH>(x, ts + i);
                        tc_wait_ld();
                    } else if (NC > CH) {
                        load(i);
                    }
#pragma unroll
                    for (int e = 0; e < CH; e += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(vf + i + e + k);
                            float2 a = __ffma2_rn(pair(x[e + k], x[e + k + 1]), cf2, nref);
                            float2 b = __ffma2_rn(pair(x[e + k + 2], x[e + k + 3]), cf2, nref);
                            a = pair(ex2f(a.x), ex2f(a.y));
                            b = pair(ex2f(b.x), ex2f(b.y));
                            sum0 = __fadd2_rn(sum0, a);
                            sum1 = __fadd2_rn(sum1, b);
                            float2 av = __fmul2_rn(a, pair(f.x, f.y)), bv = __fmul2_rn(b, pair(f.z, f.w));
                            if (nanv) {  // a V that stands for NaN does not show where it has no weight
                                av = pair(a.x == 0.0f ? 0.0f : av.x, a.y == 0.0f ? 0.0f : av.y);
                                bv = pair(b.x == 0.0f ? 0.0f : bv.x, b.y == 0.0f ? 0.0f : bv.y);
                            }
                            pk[k / 2] = pack_bf16(av.x, av.y);
                            pk[k / 2 + 1] = pack_bf16(bv.x, bv.y);
                        }
                        tc_st16(pt + (i + e) / 2, pk);
                    }
                }
                l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
                if (C > 1) {  // nothing of the other copies' keys
                    uint32_t z[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] = 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < cb / 32 || i >= (cb + NC) / 32) tc_st16(tl + kS + sb * 128 + i * 16, z);
                }
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&sh.p_full[sb]);
            }
            j = j0 + nt;
            nring += 2 * nt;
            const AttnItem done = it;
            const bool any = first < t1;                             // this group had a tile
            const int last = any ? j0 + ((t1 - 1 - first) / step) * step + (first - t0) : 0;
            u = it.u0 + it.ntiles;
            const bool more = u < uend;
            if (more) it = attn_next(p, it, items, rtiles, KT);
            if (any && ok) ok = attn_wait(&sh.pv_done[acc], (unsigned)((W == 1 ? last >> 1 : last) & 1));
            tc_fence_after();
            // the shared part's results are there, and its partial results done with
            // (no wait but after a shared pass, whose end this kernel's start overlaps)
            if (item == 0) pdl_wait_primary();
            if (W != 1) {
                auto chunk = [&](int d, float *o) {
                    tc_ld32(o, to + d);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {  // columns 0, 2, 1, 3
                        const float y = o[i + 1];
                        o[i + 1] = o[i + 2];
                        o[i + 2] = y;
                    }
                };
                attn_finish_row<T, RT, NT>(p, sh.plan, done, w, row, m, l, chunk);
            } else {
                // join the copies of both groups: 8 blocks of columns, each copy at
                // another one in each of 8 rounds (the first to come stores)
                const int g = grp * C + copy;
                sh.m[g][row] = m;
                sh.l[g][row] = l;
                sync_nt<NT>();
                float mm = -INFINITY, ll = 0.0f;
#pragma unroll
                for (int i = 0; i < K::kCopies; ++i) mm = fmaxf(mm, sh.m[i][row]);
#pragma unroll
                for (int i = 0; i < K::kCopies; ++i) ll += sh.l[i][row] * rel_weight(sh.m[i][row], mm);
                if (g == 0) {
                    sh.tm[row] = mm;
                    sh.tl[row] = ll;
                }
                const float f = rel_weight(m, mm);
                constexpr int BW = NH * 8, STEP = 8 / K::kCopies;    // columns of a block; blocks between two copies
#pragma unroll 1
                for (int h = 0; h < 8; h += 4) {
                    float o[4][BW];                                  // the blocks of four rounds
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint32_t at = to + ((g * STEP + h + s) & 7) * BW;
                        if (BW == 16) tc_ld16(o[s], at);
                        else tc_ld8(o[s], at);
                    }
                    tc_wait_ld();
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int blk = (g * STEP + h + s) & 7;
#pragma unroll
                        for (int i = 0; i < BW; i += 4) {            // columns 0, 2, 1, 3
                            float4 *at = reinterpret_cast<float4 *>(so + row * LD + blk * BW + i);
                            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (f != 0.0f) v = make_float4(o[s][i] * f, o[s][i + 2] * f, o[s][i + 1] * f, o[s][i + 3] * f);
                            if (h + s >= STEP) {
                                const float4 b = *at;
                                v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
                            }
                            *at = v;
                        }
                        sync_nt<NT>();
                    }
                }
                attn_finish<T, RT, NT>(p, sh.plan, done, w, so, LD, sh.tm, sh.tl, &sh.last);
            }
            tc_fence_before();
            mbar_arrive(&sh.q_free[qb]);
            if (!more) break;
            ++item;
        }
    }
    if (!ok && lane == 0) atomicOr(p.status, SPEC_FLAG_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tc_dealloc(tmem);
}

// ---- host ------------------------------------------------------------------
template <int NH, int C, int W> cudaError_t launch(const AttnParams &p, const CUtensorMap &cm, int sms, cudaStream_t s) {
    using K = Tc8Cfg<NH, C, W>;
    constexpr int smem = (int)sizeof(Tc8Smem<NH, C, W>) + 1024;
    static_assert(smem <= 227 * 1024 && smem > 114 * 1024, "one block an SM: it takes all of TMEM");
    static_assert(K::kRows <= kAttnSlotRows, "partial results");
    cudaError_t e = cudaFuncSetAttribute(attn8_tc_kernel<NH, C, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = sms < kAttnSmsMax ? sms : kAttnSmsMax;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(K::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = p.mode == 0 && p.P > 0 ? 1 : 0;  // after the shared pass's join
    e = cudaLaunchKernelEx(&cfg, attn8_tc_kernel<NH, C, W>, p, cm);
    return e == cudaSuccess && W != 1 ? launch_attn_join(p, K::kRows, grid, s) : e;
}

template <int NH> cudaError_t launch_nh(const AttnParams &p, const CUtensorMap &cm, int sms, cudaStream_t s) {
    const int64_t rows = p.mode == 1 ? (int64_t)p.B * p.S * p.G : (int64_t)p.S * p.G;
    if (rows <= 32) return launch<NH, 4, 1>(p, cm, sms, s);
    if (rows <= 64) return launch<NH, 2, 1>(p, cm, sms, s);
    return launch<NH, 1, 0>(p, cm, sms, s);
}

}  // namespace

// Rows of a page a box takes, as attn_tc_box; a tile's exponent bytes are read four
// at a time.
int attn8_tc_box(const AttnParams &p) {
    return reinterpret_cast<uintptr_t>(p.ks) % 4 == 0 ? attn_tc_box(p) : 0;
}

cudaError_t launch_attn8_tc(const AttnParams &p, int sms, cudaStream_t s) {
    CUtensorMap cm;
    const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.H, (cuuint64_t)(2 * p.nb * p.bs)};
    const cuuint64_t strides[2] = {(cuuint64_t)p.D, (cuuint64_t)p.H * p.D};
    const cuuint32_t box[3] = {128, 1, (cuuint32_t)p.box}, ones[3] = {1, 1, 1};
    if (tc_encode_fn()(&cm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(p.kc), dims, strides, box, ones,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return p.D <= 64 ? launch_nh<1>(p, cm, sms, s) : launch_nh<2>(p, cm, sms, s);
}

}  // namespace specv
