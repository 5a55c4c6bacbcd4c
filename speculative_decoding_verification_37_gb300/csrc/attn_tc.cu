// Attention over the paged cache for bf16 on the fifth-generation tensor cores
// (tcgen05, accumulators in TMEM; attention.cuh: score, split, join).
//
// One persistent block per SM.  A tile is 128 keys; an item's queries fill the
// 128 rows of the MMA.  Two groups of four softmax warps (a row per thread) keep
// a tile each in work:
//   * few rows (64 or 32 an item; bound by HBM): the groups take turns at the
//     tiles, with an accumulator each, and the queries are repeated C = 2 or 4
//     times down the MMA's rows.  Copy g takes only its own 128/C keys of a tile
//     (its P is zero elsewhere), so a thread has 128/C scores and no thread needs
//     another's.  The groups' and copies' results are joined at the item's end
//     like those of split keys.  The tensor work this wastes is there anyway;
//   * many rows (the pass over a shared prefix; bound by arithmetic): a query
//     tile of 128 rows for each group, both on the same keys;
//   * up to 128 rows: one group, two score tiles.
// Roles: a TMA warp copies K and V tiles, a box of a page's rows per copy, into
// a ring of buffers; one thread issues S = Q K^T and O += P V; the softmax warps
// read S from TMEM 32 columns at a time, first for the maximum, then for the
// weights, and put P, rounded to bf16, over S.  O is rescaled only when a row's
// maximum grows by more than 2^8 (the weights then stay below 2^8 of the final
// scale, well within f32 and bf16).
//
// Measured (copy rate 6.8 TB/s, cuBLAS 1,948 TFLOP/s): 64 requests of 5 queries on
// 2,048 entries of 8 heads of 128, 106 us, 5.1 TB/s; single queries on up to
// 32,768, 698 us, 6.3 TB/s; the prefix of 8,192 entries for 512 x 8 queries,
// 525 us, 1,048 TFLOP/s.  Short items are bound by what each costs alone, 6 to 9
// us: a masked last tile, the join of the copies, the division.  On the warp
// instructions (attn_mma.cu, pages of 4) the first takes 263 us, the second 1,198.
// Registers are what is short: the softmax threads use all 168, and sharing them
// out anew between the warps (88/208 to 136/184) made every case slower.
//
// A masked key's V may hold anything: where a tile masks a key, the softmax
// threads look at V's rows, one each, zero what is not finite and make NaN the
// rows that see such a key.
#include "attention.cuh"
#include "attn_tc.cuh"
#include "tma.cuh"

namespace specv {
namespace {

constexpr int KT = 128;
constexpr uint32_t kHalf = KT * 128;  // bytes: 128 keys x 64 columns
constexpr int kInfo = 8;              // tiles whose notes are kept

// Two floats an instruction (PK), or one: the pairs' registers are neighbours,
// which the kernel of two query tiles pays for with more spills (793 -> 801 us
// for 512 x 8 queries on a shared prefix; the capped tree without: 283, with: 272).
template <bool PK> __device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    return PK ? __fmul2_rn(a, b) : make_float2(a.x * b.x, a.y * b.y);
}
template <bool PK> __device__ __forceinline__ float2 add2(float2 a, float2 b) {
    return PK ? __fadd2_rn(a, b) : make_float2(a.x + b.x, a.y + b.y);
}
template <bool PK> __device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    return PK ? __ffma2_rn(a, b, c) : make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}

// How the two softmax groups share the work: W = 0 one group, 1 tiles in turn, 2
// a query tile each.
template <int NH, int C, int W> struct TcCfg {
    static constexpr int kQT = W == 2 ? 2 : 1;       // query tiles
    static constexpr int kRows = 128 * kQT / C;      // queries of an item
    static constexpr int kNT = W == 0 ? 128 : 256;   // softmax threads
    static constexpr int kThreads = kNT + (W == 2 ? 64 : 96);
    static constexpr int kQB = W == 2 ? 1 : 2;       // buffers for the queries
    static constexpr int kCopies = W == 1 ? 2 * C : C;
    static constexpr uint32_t kTile = NH * kHalf;    // bytes of a K or V tile
    // the ring takes what the queries and the join leave of 227 KB
    static constexpr int kRing = NH == 1 ? 8 : C == 2 ? 3 : 4;
};

template <int NH, int C, int W> struct TcSmem {
    using K = TcCfg<NH, C, W>;
    alignas(1024) unsigned char kv[K::kRing][K::kTile];
    alignas(1024) unsigned char q[K::kQB][K::kQT][K::kTile];
    alignas(16) float o[W == 1 ? K::kRows : 1][NH * 64 + 4];
    float m[K::kCopies][K::kRows], l[K::kCopies][K::kRows], tm[K::kRows], tl[K::kRows];
    AttnRows<K::kRows> rows[2];
    alignas(16) int kp[2][KT];      // a listed tile's keys: position,
    unsigned valid[2][4];           // whether there is such a key
    unsigned bad[kInfo];            // boxes of a tile with a bad block
    unsigned dirty[2][4];
    int low_max[2];                 // the largest first visible position of an item's rows
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

template <int NH, int C, int W, bool WH>
__global__ void __launch_bounds__(TcCfg<NH, C, W>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap cache_map,
                   const __grid_constant__ CUtensorMap temp_map) {
    using K = TcCfg<NH, C, W>;
    using T = __nv_bfloat16;
    constexpr int RT = K::kRows, NT = K::kNT, NS = K::kRing, NC = KT / C;
    constexpr int CH = W == 2 || NC < 64 ? 32 : 64;  // scores a thread holds at once (64 spill where W = 2)
    extern __shared__ unsigned char raw_[];
    TcSmem<NH, C, W> &sh = *reinterpret_cast<TcSmem<NH, C, W> *>(
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
        }
        for (int i = 0; i < K::kQB; ++i) {
            mbar_init(&sh.q_full[i], W == 2 ? NT : 32);
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
    using Lay = TcLayout<NH, WH>;
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
            const bool temp = p.tk && p.mode == 0;
            const KeyLine line = it.keys.ok ? attn_line(p, it.keys) : KeyLine{0, 0};
            const int end = temp ? it.keys.len : it.keys.hi;
            int row_k = 0, row_v = 0;      // this lane's box: row of the cache, or -1 - candidate
            auto look_up = [&](int t) {
                int r = zero_row;
                bool bad = false;
                if (lane < nbox && it.keys.ok) {
                    const int k = t * KT + lane * p.box, c = line.lo + k;
                    if (k < line.entries) {
                        if (c < end) {
                            const int j = (int)fast_div((unsigned)c, p.bs_div), blk = __ldg(table + j);
                            bad = blk < 0 || (int64_t)blk >= p.nb;
                            if (!bad) r = blk * p.bs + (c - j * p.bs);
                        }
                    } else if (temp && k - line.entries < p.S) {
                        r = -1 - (k - line.entries);
                    }
                }
                if (bad) attn_flag(p, it.b);
                const unsigned b = __ballot_sync(kFull, bad);
                if (lane == 0) sh.bad[tiles % kInfo] = b;
                ++tiles;
                return r;
            };
            auto copy = [&](int r, int is_v) {
                const int s = n % NS;
                if (n >= NS && ok) ok = attn_wait(&sh.empty[s], (unsigned)((n / NS - 1) & 1));
                if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], K::kTile);
                __syncwarp();
                if (lane < nbox) {
                    const uint32_t dst = smem_u32(sh.kv[s]) + (uint32_t)(lane * p.box >> 3) * Lay::group;
                    const int z = is_v && r >= 0 && r != zero_row ? r + v_row : r;
                    const int plane = 2 * (it.b * p.layers + p.layer) + is_v;
                    if (r < 0) {  // candidates: 8 rows and 64 columns at a time
                        for (int g = 0; g < p.box; g += 8)
#pragma unroll
                            for (int h = 0; h < NH; ++h)
                                tma4(dst + (uint32_t)(g >> 3) * Lay::group + h * Lay::half, &temp_map, h * 64, it.h, -1 - r + g,
                                     plane, &sh.full[s]);
                    } else {
                        tc_copy_box<NH, WH>(dst, &cache_map, z, it.h, &sh.full[s]);
                    }
                }
                ++n;
            };
            // the order of use: K0 K1 V0 K2 V1 ... (W = 2: K0 V0 K1 V1 ...)
            constexpr int LAG = W == 2 ? 0 : 1;
#pragma unroll 1
            for (int t = t0; t < t1 + LAG; ++t) {
                row_v = row_k;
                if (t < t1) row_k = look_up(t);
#pragma unroll 1
                for (int v = 0; v < 2; ++v)
                    if (v ? t >= t0 + LAG : t < t1) copy(v && LAG ? row_v : row_k, v);
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
            // Operands in atoms of 8 rows x 128 bytes (64 columns).  Q: the next 8
            // rows 1,024 bytes on, the next 64 columns kHalf.  K and V: Lay::group and
            // Lay::half.  16 columns of K and Q are 32 bytes; V's columns are its N,
            // contiguous (lbo: the next 64, sbo: the next 8 keys).
            constexpr uint32_t id_s = tc_idesc(KT, false), id_o = tc_idesc(NH * 64, true);
            // (one thread issues everything: an operand's descriptor is one addition.
            // Put together anew, they held the tensor cores to half their rate.)
            const uint64_t dq = tc_desc(smem_u32(sh.q[0][0]), 16, 1024), dk = tc_desc(smem_u32(sh.kv[0]), 16, Lay::group),
                           dv = tc_desc(smem_u32(sh.kv[0]), Lay::half, Lay::group);
            constexpr uint32_t k_half = Lay::half / 16, v_step = Lay::group * 2 / 16;  // V: 16 keys
            int n = 0, j = 0, item = 0;
            auto wait_full = [&](int i) {
                if (ok) ok = attn_wait(&sh.full[i % NS], (unsigned)((i / NS) & 1));
                tc_fence_after();
            };
            auto scores = [&](int d, int qt, int slot) {
                const uint64_t a = dq + (uint32_t)((item % K::kQB) * K::kQT + qt) * (K::kTile / 16), b = dk + (uint32_t)slot * (K::kTile / 16);
#pragma unroll
                for (int k = 0; k < NH * 4; ++k)
                    tc_mma_ss(tmem + kS + d * 128, a + ((k >> 2) * kHalf + (k & 3) * 32) / 16, b + (k >> 2) * k_half + (k & 3) * 32 / 16,
                              id_s, k > 0);
            };
            auto values = [&](int o, int pt, int slot, bool first) {
                const uint64_t b = dv + (uint32_t)slot * (K::kTile / 16);
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    tc_mma_ts(tmem + kO + o * 128, tmem + kS + pt * 128 + k * 8, b + k * v_step, id_o, !(first && k == 0));
            };
            auto wait_p = [&](int i, unsigned phase) {
                if (ok) ok = attn_wait(&sh.p_full[i], phase);
                tc_fence_after();
            };
            while (true) {
                const int nt = (int)(min(uend, it.u0 + it.ntiles) - u);
                if (ok) ok = attn_wait(&sh.q_full[item % K::kQB], (unsigned)((item / K::kQB) & 1));
                tc_fence_after();
                if (W != 2) {
                    // S0 S1, P0 V0, S2, P1 V1, S3 ...
                    const int j0 = j;
#pragma unroll 1
                    for (int i = 0; i < nt + 2; ++i) {
                        if (i >= 2) {
                            wait_full(n);
                            wait_p(j & 1, (unsigned)((j >> 1) & 1));
                            values(W == 0 ? 0 : j & 1, j & 1, n % NS, W == 0 ? i == 2 : i < 4);
                            tc_commit(&sh.empty[n % NS]);
                            tc_commit(&sh.pv_done[W == 0 ? 0 : j & 1]);
                            ++n;
                            ++j;
                        }
                        if (i < nt) {
                            const int d = (j0 + i) & 1;
                            wait_full(n);
                            scores(d, 0, n % NS);
                            tc_commit(&sh.empty[n % NS]);
                            tc_commit(&sh.s_full[d]);
                            ++n;
                        }
                    }
                } else {
                    wait_full(n);
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        scores(q, q, n % NS);
                        tc_commit(&sh.s_full[q]);
                    }
                    tc_commit(&sh.empty[n % NS]);
                    ++n;
#pragma unroll 1
                    for (int t = 0; t < nt; ++t, ++j) {
                        const int nv = n, nk = n + 1;
                        const bool more = t + 1 < nt;
                        wait_full(nv);
                        if (more) wait_full(nk);
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {
                            wait_p(q, (unsigned)(j & 1));
                            values(q, q, nv % NS, t == 0);
                            tc_commit(&sh.pv_done[q]);
                            if (q == 1) tc_commit(&sh.empty[nv % NS]);
                            if (more) {
                                scores(q, q, nk % NS);
                                tc_commit(&sh.s_full[q]);
                                if (q == 1) tc_commit(&sh.empty[nk % NS]);
                            }
                        }
                        n += more ? 2 : 1;
                    }
                }
                ++item;
                u = it.u0 + it.ntiles;
                if (u >= uend) break;
                it = attn_next(p, it, items, rtiles, KT);
            }
        }
        __syncwarp();
    } else if (W != 2 && warp == NT / 32 + 2) {
        // ---------------- queries ----------------
        // The next item's rows and queries, while this one's keys go by.  (W = 2
        // has no room for a second buffer: its softmax threads load them.)
        const bool by_pos = p.window > 0 || p.first != nullptr;
        const uint32_t neg = p.score.scale < 0.0f ? 0x80008000u : 0u;  // a negative scale: the queries are negated
        for (int item = 0;; ++item) {
            const int qb = item % K::kQB;
            // the buffer's last item, and its rows, are done with
            if (item >= K::kQB && ok) ok = attn_wait(&sh.q_free[qb], (unsigned)((item / K::kQB - 1) & 1));
            AttnRows<RT> &w = sh.rows[item & 1];
            attn_rows<RT, 32>(p, it, w, lane);
            __syncwarp();
            int low = (int)0x80000000;
            if (by_pos)
                for (int i = lane; i < RT; i += 32)
                    if (w.out[i] >= 0) low = max(low, max(w.first[i], p.window > 0 ? w.qp[i] - p.window + 1 : (int)0x80000000));
            low = __reduce_max_sync(kFull, low);
            if (lane == 0) sh.low_max[item & 1] = low;
            constexpr int CH = NH * 8, U = 8;  // 16-byte chunks of a row; loads in flight
#pragma unroll 1
            for (int i0 = lane; i0 < RT * CH; i0 += 32 * U) {
                uint4 v[U];
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const int i = i0 + q * 32, r = i / CH, d = (i - r * CH) * 8;
                    v[q] = make_uint4(0, 0, 0, 0);
                    if (i < RT * CH && w.q[r] >= 0 && d < p.D) v[q] = ld_nc16(static_cast<const T *>(p.q) + w.q[r] + d);
                }
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const int i = i0 + q * 32, r = i / CH, c = i - r * CH;
                    if (i >= RT * CH) continue;
                    v[q].x ^= neg, v[q].y ^= neg, v[q].z ^= neg, v[q].w ^= neg;
#pragma unroll
                    for (int k = 0; k < C; ++k) {
                        const int mr = (r + k * RT) & 127;
                        *reinterpret_cast<uint4 *>(sh.q[qb][r >> 7] + (c >> 3) * kHalf + mr * 128 + (((c & 7) ^ (mr & 7)) << 4)) = v[q];
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
        const int mrow = wq * 32 + lane;                          // row of the MMA
        const int copy = C == 1 ? 0 : wq / (4 / C);
        const int row = W == 2 ? grp * 128 + mrow : mrow % RT;    // query of the item
        const int cb = copy * NC;                                 // first key of the copy in a tile
        const int acc = W == 0 ? 0 : grp;                         // accumulator
        const int bar = W == 1 ? 2 + grp : 1, nbar = W == 1 ? 128 : NT;  // the threads that share a tile
        const uint32_t tl = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t to = tl + kO + acc * 128;
        const bool by_pos = p.window > 0 || p.first != nullptr;
        const float scale = fabsf(p.score.scale);
        int item = 0, j = 0, nring = 0;
        auto load_item = [&](const AttnItem &x, int bufn) {  // W = 2
            AttnRows<RT> &w = sh.rows[bufn];
            if (tid == 0) sh.low_max[bufn] = (int)0x80000000;
            attn_rows<RT, NT>(p, x, w, tid);
            sync_nt<NT>();
            if (by_pos && w.out[tid] >= 0)
                atomicMax(&sh.low_max[bufn], max(w.first[tid], p.window > 0 ? w.qp[tid] - p.window + 1 : (int)0x80000000));
            const uint32_t neg = p.score.scale < 0.0f ? 0x80008000u : 0u;
            constexpr int CH = NH * 8;
#pragma unroll
            for (int q = 0; q < CH; ++q) {
                const int i = tid + q * NT, r = i / CH, c = i - r * CH, d = c * 8;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (w.q[r] >= 0 && d < p.D) v = ld_nc16(static_cast<const T *>(p.q) + w.q[r] + d);
                v.x ^= neg, v.y ^= neg, v.z ^= neg, v.w ^= neg;
                const int mr = r & 127;
                *reinterpret_cast<uint4 *>(sh.q[0][r >> 7] + (c >> 3) * kHalf + mr * 128 + (((c & 7) ^ (mr & 7)) << 4)) = v;
            }
            fence_async_shared();
            mbar_arrive(&sh.q_full[0]);
        };
        if constexpr (W == 2) load_item(it, 0);
        while (true) {
            const int buf = item & 1, qb = item % K::kQB;
            if (ok) ok = attn_wait(&sh.q_full[qb], (unsigned)((item / K::kQB) & 1));
            const AttnRows<RT> &w = sh.rows[buf];
            const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0), nt = t1 - t0;
            const int qp = w.qp[row], cand = w.cand[row];
            const int low = max(w.first[row], p.window > 0 ? qp - p.window + 1 : (int)0x80000000);
            const float slope = w.slope[row];
            const bool temp = p.tk && p.mode == 0;
            const KeyLine line = it.keys.ok ? attn_line(p, it.keys) : KeyLine{0, 0};
            const int end = temp ? it.keys.len : it.keys.hi;
            float m = -INFINITY, l = 0.0f;  // reference (log2 units), sum
            bool poison = false;
            // position of key `mrow` of tile t, when key_pos is given: read a tile ahead
            auto key_pos_of = [&](int t) {
                const int k = t * KT + mrow, c = line.lo + k;
                return k < line.entries && c < it.keys.len ? __ldg(p.key_pos + (int64_t)it.b * p.kps + c) : 0;
            };
            const int step = W == 1 ? 2 : 1, first = W == 1 && (j & 1) != grp ? t0 + 1 : t0;
            int kp_next = p.key_pos && first < t1 ? key_pos_of(first) : 0;
            const int j0 = j;
            for (int t = first; t < t1; t += step) {
                const int jj = j0 + (t - t0);                      // tiles of the block so far
                const int sb = W == 0 ? jj & 1 : grp;
                const unsigned sp = W == 2 ? jj & 1 : (jj >> 1) & 1;
                const int kp_mine = kp_next;
                if (p.key_pos && t + step < t1) kp_next = key_pos_of(t + step);
                if (ok) ok = attn_wait(&sh.s_full[sb], sp);
                tc_fence_after();
                const uint32_t ts = tl + kS + sb * 128 + cb;       // this thread's scores
                const int k0 = t * KT, c0 = line.lo + k0, kb = W == 2 ? jj & 1 : W == 1 ? grp : jj & 1;
                // whether the tile may mask a key: the line's ends, candidates, a bad
                // block, the window's and the document's first tile
                const bool special = !it.keys.ok || c0 < it.keys.lo || c0 + KT > it.keys.len || k0 + KT > line.entries ||
                                     sh.bad[jj % kInfo] != 0u || (by_pos && (p.key_pos || c0 < sh.low_max[buf]));
                const bool listed = special || (p.key_pos && p.score.bias);
                // the tile's first candidate, as an index into the tile
                const int q0 = (temp ? line.entries - k0 : it.keys.len - c0);
                if (listed) {
                    if (W != 2 || grp == 0) {
                        const int k = k0 + mrow, c = c0 + mrow;
                        bool in = false;
                        int kp = 0;
                        if (it.keys.ok && k < line.entries) {
                            if (c >= it.keys.lo && c < end && !((sh.bad[jj % kInfo] >> (mrow / p.box)) & 1u)) {
                                in = true;
                                kp = c < it.keys.len ? (p.key_pos ? kp_mine : c) : key_position(p, it, c);
                            }
                        } else if (it.keys.ok && temp && k - line.entries < p.S) {
                            in = true;
                            kp = key_position(p, it, it.keys.len + k - line.entries);
                        }
                        const unsigned b = __ballot_sync(kFull, in);
                        if (lane == 0) sh.valid[kb][wq] = b;
                        sh.kp[kb][mrow] = kp;
                    }
                    bar_sync(bar, nbar);
                }
                const bool plain = !listed && p.score.cap == 0.0f && !p.score.bias;
                float x[CH];
                float cf = scale * kLog2e, mt = -INFINITY;
                bool hid = false;
                if (plain) {
#pragma unroll
                    for (int i = 0; i < NC; i += CH) {
                        tc_ldx<CH>(x, ts + i);
                        tc_wait_ld();
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
                        // (bound by issue: two scores an instruction)
                        constexpr bool PK = W != 2;
                        if (p.score.cap > 0.0f) {
                            const float ca = scale * p.score.cap_arg, c2 = -2.0f * p.score.cap;
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {  // cap_score
                                float2 v = mul2<PK>(make_float2(y[e], y[e + 1]), make_float2(ca, ca));
                                v = add2<PK>(make_float2(ex2f(v.x), ex2f(v.y)), make_float2(1.0f, 1.0f));
                                v = fma2<PK>(make_float2(rcpf(v.x), rcpf(v.y)), make_float2(c2, c2),
                                               make_float2(p.score.cap, p.score.cap));
                                y[e] = v.x, y[e + 1] = v.y;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const float2 v = mul2<PK>(make_float2(y[e], y[e + 1]), make_float2(scale, scale));
                                y[e] = v.x, y[e + 1] = v.y;
                            }
                        }
                        const int *kp = sh.kp[kb] + cb + i;
                        if (p.score.bias) {
                            const float2 ns = make_float2(-slope, -slope);
                            if (listed) {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 d = make_float2((float)pos_dist(qp, kp[e]), (float)pos_dist(qp, kp[e + 1]));
                                    const float2 v = fma2<PK>(ns, d, make_float2(y[e], y[e + 1]));
                                    y[e] = v.x, y[e + 1] = v.y;
                                }
                            } else {
                                const float d0 = (float)(qp - (c0 + cb + i));
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 d = add2<PK>(make_float2(d0, d0), make_float2((float)-e, (float)(-e - 1)));
                                    const float2 v = fma2<PK>(ns, d, make_float2(y[e], y[e + 1]));
                                    y[e] = v.x, y[e + 1] = v.y;
                                }
                            }
                        }
                        if (special) {
                            // bit e: key e of the chunk is seen by this row
                            unsigned seen = sh.valid[kb][(cb + i) / 32];
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
                            hid = hid || seen != kFull;
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
                // a masked key's V: zeros for what is not finite
                bool dirty = false;
                if (special && bar_or(bar, nbar, hid)) {
                    // V of this tile: its place in the ring by the order of the copies
                    const int tt = t - t0;
                    const int nv = nring + (W == 2 ? 2 * tt + 1 : tt + 1 < nt ? 2 * tt + 2 : 2 * tt + 1);
                    const int db = W == 1 ? grp : 0;
                    if (ok) ok = attn_wait(&sh.full[nv % NS], (unsigned)((nv / NS) & 1));
                    if (W != 2 || grp == 0) {
                        unsigned char *vr = sh.kv[nv % NS] + (mrow >> 3) * Lay::group + (mrow & 7) * 128;
                        uint32_t found = 0;
#pragma unroll 4
                        for (int i = 0; i < NH * 8; ++i) {
                            // (rows lie 128 bytes apart: neighbours start at another chunk)
                            const uint4 y = *reinterpret_cast<const uint4 *>(vr + (i >> 3) * Lay::half + ((i + lane) & 7) * 16);
                            found |= nonfinite2(y.x) | nonfinite2(y.y) | nonfinite2(y.z) | nonfinite2(y.w);
                        }
                        if (found) {
                            for (int i = 0; i < NH * 8; ++i)
                                *reinterpret_cast<uint4 *>(vr + (i >> 3) * Lay::half + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        const unsigned b = __ballot_sync(kFull, found != 0u);
                        if (lane == 0) sh.dirty[db][wq] = b;
                        if (b) fence_async_shared();
                    }
                    bar_sync(bar, nbar);
                    dirty = (sh.dirty[db][0] | sh.dirty[db][1] | sh.dirty[db][2] | sh.dirty[db][3]) != 0u;
                }
                // a new reference when the maximum has grown past 2^8 of the old one
                const bool grew = mt > m + 8.0f || (m == -INFINITY && mt > -INFINITY);
                float corr = 1.0f;
                if (grew) {
                    corr = rel_weight(m, mt);
                    m = mt;
                    l *= corr;
                }
                // (W > 0: the scores came after the product before, so O is still)
                if (__any_sync(kFull, grew) && t > first) {
                    if (W == 0) {
                        if (ok) ok = attn_wait(&sh.pv_done[0], (unsigned)((jj - 1) & 1));
                        tc_fence_after();
                    }
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
                } else if (W == 0 && t > first) {
                    // every product's end is seen before the next is let go: the
                    // barrier's phase bit tells only neighbours apart
                    if (ok) ok = attn_wait(&sh.pv_done[0], (unsigned)((jj - 1) & 1));
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                const uint32_t pt = tl + kS + sb * 128 + cb / 2;
                const float2 cf2 = make_float2(cf, cf), nref = make_float2(-ref, -ref);
                float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
                for (int i = 0; i < NC; i += CH) {
                    if (NC > CH || !plain) {
                        tc_ldx<CH>(x, ts + i);
                        tc_wait_ld();
                    }
#pragma unroll
                    for (int e = 0; e < CH; e += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            float2 a = __ffma2_rn(make_float2(x[e + k], x[e + k + 1]), cf2, nref);
                            float2 b = __ffma2_rn(make_float2(x[e + k + 2], x[e + k + 3]), cf2, nref);
                            a = make_float2(ex2f(a.x), ex2f(a.y));
                            b = make_float2(ex2f(b.x), ex2f(b.y));
                            sum0 = __fadd2_rn(sum0, a);
                            sum1 = __fadd2_rn(sum1, b);
                            pk[k / 2] = pack_bf16(a.x, a.y);
                            pk[k / 2 + 1] = pack_bf16(b.x, b.y);
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
                if (dirty) {  // a key with a non-finite V: the rows that give it weight
#pragma unroll 1
                    for (int i = 0; i < NC; i += 32) {
                        const unsigned d = sh.dirty[W == 1 ? grp : 0][(cb + i) / 32];
                        float y[16];
                        tc_ld16(y, pt + i / 2);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            poison = poison || (((d >> k) & 1u) && ((__float_as_uint(y[k / 2]) >> ((k & 1) * 16)) & 0xffffu) != 0u);
                    }
                }
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
            if (more) {
                it = attn_next(p, it, items, rtiles, KT);
                if constexpr (W == 2) load_item(it, buf ^ 1);  // (its barrier: all scores have been read)
            }
            if (any && ok)
                ok = attn_wait(&sh.pv_done[acc], (unsigned)((W == 1 ? last >> 1 : last) & 1));
            tc_fence_after();
            // the shared part's results are there, and its partial results done with
            // (no wait but after a shared pass, whose end this kernel's start overlaps)
            if (item == 0) pdl_wait_primary();
            if (W != 1) {
                auto chunk = [&](int d, float *o) {
                    tc_ld32(o, to + d);
                    tc_wait_ld();
                    if (poison)
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __int_as_float(0x7fffffff);
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
                        for (int i = 0; i < BW; i += 4) {
                            float4 *at = reinterpret_cast<float4 *>(&sh.o[row][blk * BW + i]);
                            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (f != 0.0f) v = make_float4(o[s][i] * f, o[s][i + 1] * f, o[s][i + 2] * f, o[s][i + 3] * f);
                            if (poison) v.x = v.y = v.z = v.w = __int_as_float(0x7fffffff);
                            if (h + s >= STEP) {
                                const float4 b = *at;
                                v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
                            }
                            *at = v;
                        }
                        sync_nt<NT>();
                    }
                }
                attn_finish<T, RT, NT>(p, sh.plan, done, w, &sh.o[0][0], NH * 64 + 4, sh.tm, sh.tl, &sh.last);
            }
            tc_fence_before();
            if (W != 2) mbar_arrive(&sh.q_free[qb]);
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
template <int NH, int C, int W, bool WH>
cudaError_t launch(const AttnParams &p, const CUtensorMap &cm, const CUtensorMap &tm, int sms, cudaStream_t s) {
    using K = TcCfg<NH, C, W>;
    constexpr int smem = (int)sizeof(TcSmem<NH, C, W>) + 1024;
    static_assert(smem <= 227 * 1024 && smem > 114 * 1024, "one block an SM: it takes all of TMEM");
    static_assert(K::kRows <= kAttnSlotRows * K::kQT, "partial results");
    cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<NH, C, W, WH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
    e = cudaLaunchKernelEx(&cfg, attn_tc_kernel<NH, C, W, WH>, p, cm, tm);
    return e == cudaSuccess && W != 1 ? launch_attn_join(p, K::kRows, grid, s) : e;
}

template <int NH, bool WH> cudaError_t launch_nh(const AttnParams &p, const CUtensorMap &cm, const CUtensorMap &tm, int sms, cudaStream_t s) {
    const int64_t rows = p.mode == 1 ? (int64_t)p.B * p.S * p.G : (int64_t)p.S * p.G;
    if (rows <= 32) return launch<NH, 4, 1, WH>(p, cm, tm, sms, s);
    if (rows <= 64) return launch<NH, 2, 1, WH>(p, cm, tm, sms, s);
    if (rows <= 128 || p.mode == 0) return launch<NH, 1, 0, WH>(p, cm, tm, sms, s);
    return launch<NH, 1, 2, WH>(p, cm, tm, sms, s);
}

}  // namespace

// Rows of a page a box takes: the pages must be whole boxes and a tile's 128
// keys too, 8 rows at least (a swizzle atom).
int attn_tc_box(const AttnParams &p) {
    if (p.D > 128 || 2 * p.nb * p.bs > 0x7fffff00LL || (int64_t)p.B * p.layers > 0x3fffffffLL) return 0;
    int box = 128;
    while (box >= 8 && p.bs % box != 0) box >>= 1;
    return box >= 8 && tc_encode_fn() ? box : 0;
}

cudaError_t launch_attn_tc(const AttnParams &p, int sms, cudaStream_t s) {
    CUtensorMap cm, tm;
    const cuuint64_t row = (cuuint64_t)p.H * p.D * 2;
    bool ok = tc_cache_map(p, &cm);
    tm = cm;
    if (ok && p.tk && p.mode == 0) {
        const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.H, (cuuint64_t)p.S, (cuuint64_t)p.B * p.layers * 2};
        const cuuint64_t strides[3] = {(cuuint64_t)p.D * 2, row, row * p.S};
        const cuuint32_t box[4] = {64, 1, 8, 1};
        ok = tc_encode(&tm, p.temp_base, 4, dims, strides, box);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (p.D <= 64) return launch_nh<1, true>(p, cm, tm, sms, s);
    return p.D == 128 ? launch_nh<2, true>(p, cm, tm, sms, s) : launch_nh<2, false>(p, cm, tm, sms, s);
}

}  // namespace specv
