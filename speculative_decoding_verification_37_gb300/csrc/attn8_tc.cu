// Attention over the 8-bit paged cache for bf16 queries on the fifth-generation
// tensor cores (attention.cuh: score, split, join; kv8.cuh: the cache's numbers).
//
// One persistent block per SM, in three teams that know nothing of each other: a team
// has a warp that copies, four softmax warps and its own share of the line of tiles
// (one warp issues the MMAs of all), so that what one waits for (a product's end, an
// item's first keys, its output) the others' work covers.  A tile is 128 keys, down
// the MMA's rows; an item's 16 or 32 queries are its columns: a thread has a key,
// with the key's power of two, position and masks, and the MMA does no work for
// queries that are not there.  K and V go to the tensor cores as the codes they are:
//   * S^T = K Q^T.  A query, scaled by a power of two, is the sum of two e4m3 numbers
//     (8 significant bits, as bf16 has; the smallest elements may lose 2^-17 of the
//     largest); both products go into one accumulator.  A key's power of two
//     multiplies its scores.
//   * O^T = V^T P^T.  A weight of 2^-20 next to one of 1 is worth keeping where there are
//     many, and e4m3 ends at 2^-9.  So a weight, times its key's power of two relative
//     to the largest that the row has seen, is rounded to f16 and taken apart into three
//     e5m2 numbers: the upper byte of an f16 is one, and what it leaves is an f16
//     again.  So the parts cost an AND, a subtraction and half a byte shuffle each, need
//     no scales, and hold 9 bits, or 2^-24 of a weight of 1 at the largest power.  They are
//     columns of one product and are added at the item's end.
//   * A row's largest score lies across the threads.  It is looked for, and the
//     largest power, in an item's first tile and where a score passes the reference
//     by 2^8 or a power the smallest of the rows', which one vote of the tile's threads
//     finds; otherwise nobody needs another's scores.  Tiles go from the last, which is
//     full, to the first: with a bias by distance the largest scores come first.  Sums
//     of weights stay in the threads until the item's end.
//   * Where a tile hides keys, the threads look whether V holds NaN's code: such a row
//     becomes zeros and gives its NaN, by way of the power of two, to the rows that
//     give it weight; the rows that it is hidden from see nothing.
#include <cuda_fp16.h>

#include "attention.cuh"
#include "attn_tc.cuh"
#include "kv8.cuh"
#include "tma.cuh"

namespace specv {
namespace {

constexpr int KT = 128, GT = 128, NT = 256;  // keys of a tile; softmax threads of a team; threads that plan
constexpr uint32_t kTile = KT * 128;  // bytes of 128 keys x up to 128 codes
constexpr int kInfo = 4;              // tiles whose notes are kept
constexpr float kNone = -1e30f;       // the reference of a row that has seen no key
constexpr float kLag = 8.0f;          // log2 of what a weight may reach
constexpr int kPowMin = 16;           // exponent byte that smaller powers are taken relative to
constexpr int kUp = 7;                // log2 of a weight of 1 at the largest power: 2^(kUp + kLag) is an e5m2 number
constexpr int kParts = 3;             // e5m2 numbers that hold a weight

__device__ __forceinline__ float2 pair(float a, float b) { return make_float2(a, b); }

// e4m3 x e4m3 -> f32, M = 128, both operands K-major
__host__ __device__ constexpr uint32_t tc_idesc8(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24); }
// e4m3 x e5m2, both operands' rows contiguous
__host__ __device__ constexpr uint32_t tc_idesc_mn(int n) { return tc_idesc8(n) | (1u << 10) | (1u << 15) | (1u << 16); }
__device__ __forceinline__ void tc_mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
template <int N> __device__ __forceinline__ void tc_load(float *x, uint32_t t) {
    if (N == 16) tc_ld16(x, t);
    else tc_ldx<N>(x, t);
}
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

// Shared-memory operands: 64- and 32-byte swizzles (8 rows of so many bytes an atom)
__device__ __forceinline__ uint64_t tc_desc64(uint32_t addr, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (4ull << 61);
}
__device__ __forceinline__ uint64_t tc_desc32(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (6ull << 61);
}
// whether a barrier's phase is over; waits for nothing
__device__ __forceinline__ bool mbar_test(unsigned long long *bar, unsigned phase) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(phase)
        : "memory");
    return ok != 0u;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two f16, which lose their upper bytes: what e5m2 numbers of them leave.
__device__ __forceinline__ uint32_t rest_e5m2(uint32_t h) {
    const uint32_t top = h & 0xff00ff00u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&top));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t round_e5m2(uint32_t h) {
    uint16_t c;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
    return c;
}
// 2^e of -126 <= e <= 127; below: 0
__device__ __forceinline__ float pow2i(int e) { return e < -126 ? 0.0f : __uint_as_float((unsigned)(e + 127) << 23); }

// the warp's largest, a NaN left out
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
// op over the warp's lanes of each of N rows' values: lane i has the result of row i
// (N = 16: of row i / 2) in v[0].
template <int N, typename F> __device__ __forceinline__ void reduce_rows(float (&v)[N], F &&op) {
    const int lane = threadIdx.x & 31;
    int n = N;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
                    v[i] = op(keep, __shfl_xor_sync(kFull, give, o));
                }
        } else {
            v[0] = op(v[0], __shfl_xor_sync(kFull, v[0], o));
        }
    }
}

constexpr int kTeams = 3;

// What a team has.
template <int NH, int RT> struct Team8 {
    static constexpr uint32_t kQ = RT * 128;         // bytes of a part of the queries
    // P^T: 16 queries: a key's 64 bytes, three parts of four; 32: a part's 4 KB after another
    static constexpr uint32_t kP = RT == 16 ? KT * 64 : KT * kParts * 32, kStep = RT == 16 ? 32 * 64 : 32 * 32;
    static constexpr int KS = 2;                     // buffers for K
    alignas(1024) unsigned char k[KS][kTile];
    alignas(1024) unsigned char v[kTile];
    alignas(1024) unsigned char q[2][kQ];            // the queries' first and second parts
    alignas(1024) unsigned char p[kP];
    alignas(16) float ref[RT], corr[RT], corr_o[RT], gain[RT];  // references (log2 units), what sums and O are
                                                     // multiplied by, what weights are at a power of 1
    alignas(16) float top[4][RT];                    // the warps' largest scores; at the end sums of weights
    alignas(16) int pow[4][RT];                      // and powers
    alignas(16) float cf[RT];                        // scale times what the queries were divided by; without cap and bias times log2(e)
    alignas(16) float qp[RT];                        // positions after the item's first
    alignas(16) int low[RT];                         // first visible position
    alignas(16) float fa[RT], fc[RT];                // output: factors of O and of the shared part
    AttnRows<RT> rows[2];
    unsigned words[RT][5];                           // a tile's candidates in the rows' tree masks
    int pow_min, low_max, qp0;                       // the smallest largest power; the largest `low`; the first position
    unsigned sc[kInfo][2][KT / 4];                   // exponent bytes of a tile's K and V
    unsigned bad[kInfo];                             // boxes of a tile with a bad block
    int first[kInfo];                                // whether an item begins
    alignas(8) unsigned long long k_full[KS], k_empty[KS], v_full, s_full[2], p_full, pv_done, q_full;
    int scored, weighed, begun, tiles;               // the MMA warp's: tiles so far, items begun, tiles in all
    int last;
};
template <int NH, int RT> struct Tc8Smem {
    Team8<NH, RT> team[kTeams];
    AttnPlan plan;
    uint32_t tmem;
};

// the item after `it` (one copy of this code)
static __device__ __noinline__ void next_item(const AttnParams &p, AttnItem &it, int items, int rtiles) {
    it = attn_next(p, it, items, rtiles, KT);
}
// The first key of an item's line of tiles: the last tile is full, the first has what
// is left (whole boxes).
__device__ __forceinline__ int line_start(const KeyLine &line, int ntiles) { return line.lo - (ntiles * KT - line.entries); }

template <int NH, int RT, bool plain>
__global__ void __launch_bounds__(128 * kTeams + 128, 1)
    attn8_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap cache_map) {
    using H = Team8<NH, RT>;
    constexpr int G = kTeams, NW = 4 * G;  // teams; softmax warps
    using T = __nv_bfloat16;
    extern __shared__ unsigned char raw_[];
    Tc8Smem<NH, RT> &all = *reinterpret_cast<Tc8Smem<NH, RT> *>(
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw_) + 1023) & ~uintptr_t(1023)));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = warp < NW ? warp >> 2 : warp < NW + G ? warp - NW : 0;  // then a warp a team for copies, one for MMAs
    H &sh = all.team[grp];
    const int per = p.S * p.G;
    const int64_t nrows = p.mode == 1 ? (int64_t)p.B * per : per;
    const int rtiles = (int)((nrows + RT - 1) / RT), items = p.H * rtiles;
    if (tid < G) {
        H &h = all.team[tid];
        for (int s = 0; s < H::KS; ++s) {
            mbar_init(&h.k_full[s], 1);
            mbar_init(&h.k_empty[s], 1);
        }
        mbar_init(&h.v_full, 1);
        mbar_init(&h.s_full[0], 1);
        mbar_init(&h.s_full[1], 1);
        mbar_init(&h.p_full, GT);
        mbar_init(&h.pv_done, 1);
        mbar_init(&h.q_full, GT);
        fence_barrier_init();
    }
    if (p.mode == 1) pdl_launch_dependents();  // (they wait before they use what this kernel writes)
    if (warp < NT / 32) attn_plan<NT>(p, all.plan, items, KT);
    if (warp == NW) tc_alloc(&all.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = all.tmem;
    // A team's share of the line; the first teams have its first part, so that few
    // tiles lie on many SMs.
    const int64_t parts = G * (int64_t)gridDim.x, share = (all.plan.total + parts - 1) / parts;
    const int part = grp * (int)gridDim.x + (int)blockIdx.x;
    int64_t u = part * share;
    const int64_t uend = min(all.plan.total, u + share);
    // TMEM columns: the teams' two score tiles, then their accumulators
    constexpr uint32_t kO = 2 * G * RT;
    const uint32_t col_s = tmem + grp * 2 * RT, col_o = tmem + kO + kParts * grp * RT;
    static_assert((2 + kParts) * G * RT <= 512, "columns");
    bool ok = true;  // after a wait has run out nothing waits any more; the call is flagged
    if (warp == NW + G) {
        // ---------------- MMAs ----------------
        // A team's next product where its weights and V are there, its next scores where its
        // K is, and, of an item's first, the queries.
        if (lane == 0) {
            // Operands.  Scores: atoms of 8 rows x 128 bytes, the next 8 rows 1,024 bytes on;
            // 32 columns of K and Q are 32 bytes.  Values: the rows are keys, the products' K,
            // whose elements (V's columns: M; P's weights: N) are contiguous: 128 of V (zeros
            // past the head), 48 of P, or 32 and the next 32 a part further on.
            constexpr uint32_t id_s = tc_idesc8(RT), id_o = tc_idesc_mn(kParts * RT);
            int left = 0, idle = 0;
            for (int g = 0; g < G; ++g) {
                H &t = all.team[g];
                const int64_t at = ((int64_t)g * gridDim.x + blockIdx.x) * share;
                t.scored = t.weighed = t.begun = 0;
                left += t.tiles = (int)max((int64_t)0, min(all.plan.total, at + share) - at);
            }
            while (left > 0 && idle < (int)kSpinLimit) {
                ++idle;
#pragma unroll 1
                for (int g = 0; g < G; ++g) {
                    H &t = all.team[g];
                    const int n = t.scored, j = t.weighed;
                    if (j < n && mbar_test(&t.v_full, (unsigned)(j & 1)) && mbar_test(&t.p_full, (unsigned)(j & 1))) {
                        tc_fence_after();
                        const uint64_t a = tc_desc(smem_u32(t.v), 0, 1024),
                                       b = RT == 16 ? tc_desc64(smem_u32(t.p), 512) : tc_desc32(smem_u32(t.p), KT * 32, 256);
                        const bool add = !t.first[j % kInfo];
#pragma unroll
                        for (int k = 0; k < KT / 32; ++k)
                            tc_mma8(tmem + kO + kParts * g * RT, a + k * (4096 / 16), b + k * (H::kStep / 16), id_o, add || k > 0);
                        tc_commit(&t.pv_done);
                        t.weighed = j + 1;
                        --left;
                        idle = 0;
                    }
                    if (n < t.tiles && n < t.weighed + 2 && mbar_test(&t.k_full[n % H::KS], (unsigned)((n / H::KS) & 1))) {
                        const bool first = t.first[n % kInfo];
                        if (!first || mbar_test(&t.q_full, (unsigned)(t.begun & 1))) {
                            tc_fence_after();
                            const uint64_t a = tc_desc(smem_u32(t.k[n % H::KS]), 16, 1024), b = tc_desc(smem_u32(t.q[0]), 16, 1024);
#pragma unroll
                            for (int k = 0; k < NH * 4; ++k)  // first parts, second parts
                                tc_mma8(tmem + (2 * g + (n & 1)) * RT, a + (k % (NH * 2)) * (32 / 16),
                                        b + (k / (NH * 2)) * (H::kQ / 16) + (k % (NH * 2)) * (32 / 16), id_s, k > 0);
                            tc_commit(&t.k_empty[n % H::KS]);
                            tc_commit(&t.s_full[n & 1]);
                            t.scored = n + 1;
                            t.begun += first;
                            idle = 0;
                        }
                    }
                }
            }
            ok = left == 0;
        }
        __syncwarp();
    } else if (u < uend) {
        AttnItem it = attn_find<NT>(p, all.plan, u, items, rtiles, KT);
        if (warp >= NW) {
            // ---------------- copies ----------------
            const int nbox = KT / p.box;
            const int zero_row = (int)(2 * p.nb * p.bs);  // past the map: zeros are written
            const int v_row = (int)(p.nb * p.bs);
            int n = 0;
            while (true) {
                if (!it.keys.ok && u == it.u0 && it.h == 0 && it.rt == 0 && lane == 0) attn_flag(p, it.b);
                const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
                const int *table = p.mode == 1 ? p.stable : p.table + (int64_t)it.b * p.max_blocks;
                const KeyLine line = it.keys.ok ? attn_line(p, it.keys) : KeyLine{0, 0};
                // A lane looks up 4 keys (a page has a multiple of 8): their block two tiles
                // ahead, their exponents one; a box's row comes from the lane that has its
                // first key.
                int blk = 0, row = 0;
                unsigned ks = 0u, vs = 0u;
                bool bad = false;
                const int start = line_start(line, it.ntiles);
                auto has = [&](int t) {
                    const int c = start + t * KT + lane * 4;
                    return t >= t0 && it.keys.ok && c >= line.lo && c < it.keys.hi;
                };
                auto block_of = [&](int t) {
                    return has(t) ? __ldg(table + fast_div((unsigned)(start + t * KT + lane * 4), p.bs_div)) : 0;
                };
                auto entry_of = [&](int t) {
                    ks = vs = 0u;
                    row = zero_row;
                    bad = false;
                    if (has(t)) {
                        const int c = start + t * KT + lane * 4, at = c - (int)fast_div((unsigned)c, p.bs_div) * p.bs;
                        bad = blk < 0 || (int64_t)blk >= p.nb;
                        if (!bad) {
                            row = blk * p.bs + at;
                            const int64_t s = ((int64_t)blk * p.H + it.h) * p.bs + at;
                            ks = __ldg(reinterpret_cast<const unsigned *>(p.ks + s));
                            vs = __ldg(reinterpret_cast<const unsigned *>(p.vs + s));
                        }
                    }
                };
                auto copy = [&](unsigned char *to, unsigned long long *bar, int r) {
                    if (lane == 0) mbar_arrive_expect_tx(bar, kTile);
                    __syncwarp();
                    if (lane < nbox) tma3(smem_u32(to) + (uint32_t)(lane * p.box) * 128u, &cache_map, 0, it.h, r, bar);
                };
                blk = block_of(t1 - 1);
                entry_of(t1 - 1);
                blk = block_of(t1 - 2);
                int box_v = 0;
                // the order of use: K0 K1 V0 K2 V1 ...
#pragma unroll 1
                for (int t = t1 - 1; t >= t0 - 1; --t) {
                    const int box_before = box_v;
                    if (t >= t0) {
                        if (bad) attn_flag(p, it.b);
                        const int from = lane < nbox ? lane * p.box >> 2 : 0, i = n % kInfo, s = n % H::KS;
                        const bool box_bad = __shfl_sync(kFull, (int)bad, from) != 0;
                        const int box = __shfl_sync(kFull, row, from);
                        const unsigned b = __ballot_sync(kFull, box_bad && lane < nbox);
                        if (n >= H::KS && ok) ok = attn_wait(&sh.k_empty[s], (unsigned)((n / H::KS - 1) & 1));
                        sh.sc[i][0][lane] = ks;
                        sh.sc[i][1][lane] = vs;
                        if (lane == 0) {
                            sh.bad[i] = b;
                            sh.first[i] = t == t1 - 1;
                        }
                        __syncwarp();  // (the notes, before the arrival)
                        copy(sh.k[s], &sh.k_full[s], box);
                        box_v = box == zero_row ? box : box + v_row;
                        entry_of(t - 1);
                        blk = block_of(t - 2);
                        ++n;
                    }
                    if (t < t1 - 1) {
                        const int j = n - (t >= t0 ? 2 : 1);
                        if (j > 0 && ok) ok = attn_wait(&sh.pv_done, (unsigned)((j - 1) & 1));
                        __syncwarp();
                        copy(sh.v, &sh.v_full, box_before);
                    }
                }
                u = it.u0 + it.ntiles;
                if (u >= uend) break;
                next_item(p, it, items, rtiles);
            }
            // no copy may land after the block has gone
            for (int i = max(0, n - H::KS); i < n; ++i) ok = mbar_drain(&sh.k_full[i % H::KS], (unsigned)((i / H::KS) & 1)) && ok;
            ok = mbar_drain(&sh.v_full, (unsigned)((n - 1) & 1)) && ok;
        } else {
            // ---------------- softmax ----------------
            const int wq = warp & 3, key = tid & (GT - 1);            // key of a tile; row of the MMA: TMEM lane
            const int bar = 2 + grp;
            const uint32_t lanes = (uint32_t)(wq * 32) << 16;
            const uint32_t to = col_o + lanes;
            const bool by_pos = p.window > 0 || p.first != nullptr;
            const uint32_t neg = p.score.scale < 0.0f ? 0x80008000u : 0u;  // a negative scale: the queries are negated
            const float scale = fabsf(p.score.scale) * (plain ? kLog2e : 1.0f);
            constexpr unsigned kRowLanes = RT == 16 ? 0xffffu : kFull;
            int item = 0, n = 0;
            auto start_rows = [&] {  // of an item: nothing seen yet
                if (key < RT) {
                    sh.ref[key] = kNone;
                    sh.gain[key] = pow2i(127 + kUp - kPowMin);
                }
            };
            // An item's rows and queries: 8 elements a thread at a time.  The next item's are
            // prepared before this one's output.
            auto prepare = [&](AttnRows<RT> &w) {
                attn_rows<RT, GT>(p, it, w, key);
                if (key < RT) {
                    const int lo = max(w.first[key], p.window > 0 ? w.qp[key] - p.window + 1 : (int)0x80000000);
                    sh.low[key] = lo;
                    const bool is = w.out[key] >= 0;
                    const int most = __reduce_max_sync(kRowLanes, is ? lo : (int)0x80000000);
                    const int qp0 = __reduce_min_sync(kRowLanes, is ? w.qp[key] : 0x7fffffff);
                    sh.qp[key] = is ? (float)pos_dist(w.qp[key], qp0) : 0.0f;
                    if (lane == 0) {
                        sh.low_max = most;
                        sh.qp0 = qp0;
                    }
                }
                bar_sync(bar, GT);
                constexpr int LR = NH * 8, Q = RT * LR / GT;          // lanes of a row; a thread's pieces
                const int d = (key % LR) * 8;
                uint4 v[Q];
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const int r = key / LR + i * (GT / LR);
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (w.q[r] >= 0 && d < p.D) v[i] = ld_nc16(static_cast<const T *>(p.q) + w.q[r] + d);
                }
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const int r = key / LR + i * (GT / LR);
                    v[i].x ^= neg, v[i].y ^= neg, v[i].z ^= neg, v[i].w ^= neg;
                    float x[8], top = 0.0f;
                    unpack<T>(v[i], x);
                    if (nonfinite2(v[i].x) | nonfinite2(v[i].y) | nonfinite2(v[i].z) | nonfinite2(v[i].w)) top = INFINITY;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
                    for (int o = LR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
                    const unsigned s = kv8_scale(top);
                    const float f = s == 255u ? 0.0f : kv8_inverse(s);
                    if (key % LR == 0) sh.cf[r] = scale * kv8_power(s);
                    uint32_t a[2], b[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        a[e] = kv8_code2(x[4 * e] * f, x[4 * e + 1] * f) | kv8_code2(x[4 * e + 2] * f, x[4 * e + 3] * f) << 16;
                        const float4 y = kv8_value4(a[e]);
                        b[e] = kv8_code2(x[4 * e] * f - y.x, x[4 * e + 1] * f - y.y) |
                               kv8_code2(x[4 * e + 2] * f - y.z, x[4 * e + 3] * f - y.w) << 16;
                    }
                    const uint32_t at = r * 128 + (((d >> 4) ^ (r & 7)) << 4) + (d & 8);
                    *reinterpret_cast<uint2 *>(sh.q[0] + at) = make_uint2(a[0], a[1]);
                    *reinterpret_cast<uint2 *>(sh.q[1] + at) = make_uint2(b[0], b[1]);
                }
                fence_async_shared();
                bar_sync(bar, GT);
                mbar_arrive(&sh.q_full);
            };
            start_rows();
            prepare(sh.rows[0]);
            while (true) {
                const AttnRows<RT> &w = sh.rows[item & 1];
                const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
                const KeyLine line = it.keys.ok ? attn_line(p, it.keys) : KeyLine{0, 0};
                const int start = line_start(line, it.ntiles);
                const int low_max = sh.low_max, qp0 = sh.qp0;
                int pow_min = 0;                 // the smallest of the rows' largest powers
                float l[RT];                     // sums of this thread's weights
#pragma unroll
                for (int r = 0; r < RT; ++r) l[r] = 0.0f;
                // position of this thread's key of tile t, when key_pos is given: read a tile ahead
                auto key_pos_of = [&](int t) {
                    const int c = start + t * KT + key;
                    return it.keys.ok && c >= line.lo && c < it.keys.len ? __ldg(p.key_pos + (int64_t)it.b * p.kps + c) : 0;
                };
                int kp_next = p.key_pos ? key_pos_of(t1 - 1) : 0;
                const int n0 = n;
#pragma unroll 1
                for (int t = t1 - 1; t >= t0; --t, ++n) {
                    const int c0 = start + t * KT;
                    int kp = c0 + key;
                    if (p.key_pos) {
                        kp = kp_next;
                        if (t > t0) kp_next = key_pos_of(t - 1);
                    }
                    if (ok) ok = attn_wait(&sh.s_full[n & 1], (unsigned)((n >> 1) & 1));
                    tc_fence_after();
                    // (the tile's notes were there before its K)
                    const unsigned char *sc = reinterpret_cast<const unsigned char *>(sh.sc[n % kInfo][0]);
                    const float kf = kv8_power(sc[key]);
                    const int vs = sc[KT + key], pw = vs == 255 ? 0 : vs;
                    const unsigned bad = sh.bad[n % kInfo];
                    // whether the tile may mask a key: the line's ends, candidates, a bad
                    // block, the window's and the document's first tile
                    const bool special = !it.keys.ok || c0 < it.keys.lo || c0 + KT > it.keys.len ||
                                         bad != 0u || (by_pos && (p.key_pos || c0 < low_max));
                    const int cand = c0 + key - it.keys.len;           // the key as a candidate, or < 0
                    bool in = true;
                    if (special) {
                        in = it.keys.ok && c0 + key >= it.keys.lo && c0 + key < it.keys.hi &&
                             !((bad >> (key / p.box)) & 1u);
                        if (in && cand >= 0) kp = key_position(p, it, c0 + key);
                    }
                    unsigned seen = kFull;                             // bit r: by row r
                    if (special) {
                        // (the tree masks' words of a tile with candidates: loaded once, by the rows)
                        const bool tree = p.mode == 0 && p.mask && c0 + KT > it.keys.len;
                        const int word0 = max(c0 - it.keys.len, 0) >> 5;
                        if (tree) {
                            for (int i = key; i < RT * 5; i += GT) {
                                const int r = i / 5, x = word0 + i - r * 5;
                                sh.words[r][i - r * 5] = x < p.W ? p.mask[((int64_t)it.b * p.S + w.cand[r]) * p.W + x] : 0u;
                            }
                            bar_sync(bar, GT);
                        }
                        if (!in) {
                            seen = 0u;
                        } else if (by_pos || (p.mode == 0 && cand >= 0)) {
                            const int x = (cand >> 5) - word0;
                            seen = 0u;
#pragma unroll 8
                            for (int r = 0; r < RT; ++r) {
                                bool s = !by_pos || kp >= sh.low[r];
                                if (p.mode == 0 && cand >= 0) s = s && (tree ? (sh.words[r][x] >> (cand & 31)) & 1u : cand <= w.cand[r]);
                                seen |= (unsigned)s << r;
                            }
                        }
                    }
                    const uint32_t ts = col_s + (n & 1) * RT + lanes;
                    const float kd = (float)pos_dist(qp0, kp);
                    // Scores in log2 units less the references; without them (raw) to find new ones.
                    float y[RT];
                    bool raw = n == n0;
#pragma unroll 1
                    while (true) {
                        tc_load<RT>(y, ts);
                        tc_wait_ld();
                        const float2 kf2 = pair(kf, kf), e2 = pair(kLog2e, kLog2e);
#pragma unroll
                        for (int r = 0; r < RT; r += 4) {  // (the key's factor first: with the query's it is the score's size)
                            const float2 a = __fmul2_rn(pair(y[r], y[r + 1]), kf2), b = __fmul2_rn(pair(y[r + 2], y[r + 3]), kf2);
                            y[r] = a.x, y[r + 1] = a.y, y[r + 2] = b.x, y[r + 3] = b.y;
                        }
                        if (!plain) {
                            if (p.score.cap > 0.0f) {  // cap_score
                                const float2 s2 = pair(p.score.cap_arg, p.score.cap_arg), c2 = pair(-2.0f * p.score.cap, -2.0f * p.score.cap),
                                             cap2 = pair(p.score.cap, p.score.cap), one = pair(1.0f, 1.0f);
#pragma unroll
                                for (int r = 0; r < RT; r += 2) {
                                    float2 a = __fmul2_rn(__fmul2_rn(pair(y[r], y[r + 1]), *reinterpret_cast<const float2 *>(&sh.cf[r])), s2);
                                    a = __fadd2_rn(pair(ex2f(a.x), ex2f(a.y)), one);
                                    a = __ffma2_rn(pair(rcpf(a.x), rcpf(a.y)), c2, cap2);
                                    y[r] = a.x, y[r + 1] = a.y;
                                }
                            } else {
#pragma unroll
                                for (int r = 0; r < RT; r += 2) {
                                    const float2 a = __fmul2_rn(pair(y[r], y[r + 1]), *reinterpret_cast<const float2 *>(&sh.cf[r]));
                                    y[r] = a.x, y[r + 1] = a.y;
                                }
                            }
                            if (p.score.bias) {  // (both terms of the distance are positive for entries: no cancellation)
                                const float2 kd2 = pair(kd, kd);
#pragma unroll
                                for (int r = 0; r < RT; r += 2) {
                                    const float2 d = __fadd2_rn(*reinterpret_cast<const float2 *>(&sh.qp[r]), kd2);
                                    const float2 s = *reinterpret_cast<const float2 *>(&w.slope[r]);
                                    const float2 a = __ffma2_rn(pair(-s.x, -s.y), d, pair(y[r], y[r + 1]));
                                    y[r] = a.x, y[r + 1] = a.y;
                                }
                            }
                        }
#pragma unroll
                        for (int r = 0; r < RT; r += 4) {
                            const float4 m = raw ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4 *>(&sh.ref[r]);
                            const float4 c = plain ? *reinterpret_cast<const float4 *>(&sh.cf[r]) : make_float4(kLog2e, kLog2e, kLog2e, kLog2e);
                            const float2 a = __ffma2_rn(pair(y[r], y[r + 1]), pair(c.x, c.y), pair(-m.x, -m.y));
                            const float2 b = __ffma2_rn(pair(y[r + 2], y[r + 3]), pair(c.z, c.w), pair(-m.z, -m.w));
                            y[r] = a.x, y[r + 1] = a.y, y[r + 2] = b.x, y[r + 3] = b.y;
                        }
                        if (special) {
#pragma unroll
                            for (int r = 0; r < RT; ++r) y[r] = (seen >> r) & 1u ? y[r] : -INFINITY;
                        }
                        if (!raw) {
                            const float over = max_of<RT>(y);
                            if (!bar_or(bar, GT, over > kLag || (in && pw > pow_min))) break;
                            raw = true;
                            continue;
                        }
                        // The tile's largest scores and powers; a new reference where a row's score
                        // has grown past 2^kLag of the old one.
                        float mine = -INFINITY;  // of row `lane`
                        int most = 0;
                        const int every = __reduce_max_sync(kFull, pw);
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const float m = warp_max(y[r]);
                            if (lane == r) mine = m;
                        }
                        if (special) {
#pragma unroll 8
                            for (int r = 0; r < RT; ++r) {
                                const int m = __reduce_max_sync(kFull, (seen >> r) & 1u ? pw : 0);
                                if (lane == r) most = m;
                            }
                        } else {  // every row sees every key
                            most = every;
                        }
                        if (lane < RT) {
                            sh.top[wq][lane] = mine;
                            sh.pow[wq][lane] = most;
                        }
                        bar_sync(bar, GT);
                        if (key < RT) {
                            const float top = fmaxf(fmaxf(sh.top[0][key], sh.top[1][key]), fmaxf(sh.top[2][key], sh.top[3][key]));
                            const int most = max(max(sh.pow[0][key], sh.pow[1][key]), max(sh.pow[2][key], sh.pow[3][key]));
                            const float old = sh.ref[key];
                            const bool grew = top > old + kLag || (old == kNone && top > kNone);
                            const float f = grew ? ex2f(old - top) : 1.0f;
                            const int was = 127 + kUp - ((int)(__float_as_uint(sh.gain[key]) >> 23) - 127), now = max(was, most);
                            sh.corr[key] = f;
                            sh.corr_o[key] = f * pow2i(was - now);
                            sh.gain[key] = pow2i(127 + kUp - now);
                            if (grew) sh.ref[key] = top;
                            const int least = __reduce_min_sync(kRowLanes, grew || old != kNone ? now : 254);
                            if (lane == 0) sh.pow_min = least;
                        }
                        bar_sync(bar, GT);
                        pow_min = sh.pow_min;
#pragma unroll
                        for (int r = 0; r < RT; r += 4) {
                            const float4 m = *reinterpret_cast<const float4 *>(&sh.ref[r]), f = *reinterpret_cast<const float4 *>(&sh.corr[r]);
                            y[r] -= m.x, y[r + 1] -= m.y, y[r + 2] -= m.z, y[r + 3] -= m.w;
                            l[r] *= f.x, l[r + 1] *= f.y, l[r + 2] *= f.z, l[r + 3] *= f.w;
                        }
                        if (n > n0) {  // O, still once the product before has ended
                            if (ok) ok = attn_wait(&sh.pv_done, (unsigned)((n - 1) & 1));
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < kParts * RT; c += 16) {
                                const float *f = sh.corr_o + (c & (RT - 1));
                                float o[16];
                                uint32_t z[16];
                                tc_ld16(o, to + c);
                                tc_wait_ld();
#pragma unroll
                                for (int r = 0; r < 16; ++r) z[r] = __float_as_uint(o[r] * f[r]);
                                tc_st16(to + c, z);
                            }
                            tc_wait_st();
                        }
                        break;
                    }
                    float vf = kv8_power(vs);
                    if (special) {
                        // V's NaN must not meet the weights of rows that do not see it
                        if (ok) ok = attn_wait(&sh.v_full, (unsigned)(n & 1));
                        unsigned char *vr = sh.v + key * 128;
                        uint32_t nan = 0;
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {  // (neighbours start at another chunk)
                            const uint4 c = *reinterpret_cast<const uint4 *>(vr + (((i + lane) & 7) << 4));
                            nan |= ((c.x & 0x7f7f7f7fu) + 0x01010101u) | ((c.y & 0x7f7f7f7fu) + 0x01010101u) |
                                   ((c.z & 0x7f7f7f7fu) + 0x01010101u) | ((c.w & 0x7f7f7f7fu) + 0x01010101u);
                        }
                        if (nan & 0x80808080u) {
                            vf = kv8_power(255);
#pragma unroll 1
                            for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(vr + (i << 4)) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    // P's buffer is free once the product before has ended
                    if (n > n0 && ok) ok = attn_wait(&sh.pv_done, (unsigned)((n - 1) & 1));
                    // weights: summed, times V's power of two to three e4m3 numbers
                    unsigned char *pp = sh.p + key * (RT == 16 ? 64 : 32);
                    const int sw = RT == 16 ? (key >> 1) & 3 : (key >> 2) & 1;  // the swizzle of 64 or 32 bytes
                    const bool pick = special || vf != vf;
#pragma unroll
                    for (int r = 0; r < RT; r += 16) {
                        uint32_t h[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int q = r + 2 * i;
                            const float2 g = *reinterpret_cast<const float2 *>(&sh.gain[q]);
                            const float2 a = pair(ex2f(y[q]), ex2f(y[q + 1]));
                            const float2 sum = __fadd2_rn(pair(l[q], l[q + 1]), a);
                            l[q] = sum.x, l[q + 1] = sum.y;
                            float2 b = __fmul2_rn(a, __fmul2_rn(g, pair(vf, vf)));
                            // (a V that stands for NaN does not show where it has no weight; a hidden
                            // one's power may be any)
                            if (pick) b = pair(a.x == 0.0f ? 0.0f : b.x, a.y == 0.0f ? 0.0f : b.y);
                            h[i] = pack_f16(b.x, b.y);
                        }
                        auto put = [&](int c) {
                            uint32_t z[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) z[i] = c < 2 ? __byte_perm(h[2 * i], h[2 * i + 1], 0x7531) : h[2 * i] | h[2 * i + 1] << 16;
                            *reinterpret_cast<uint4 *>(pp + (RT == 16 ? (c ^ sw) << 4 : c * (KT * 32) + ((r / 16 ^ sw) << 4))) = make_uint4(z[0], z[1], z[2], z[3]);
                        };
                        put(0);
#pragma unroll
                        for (int i = 0; i < 8; ++i) h[i] = rest_e5m2(h[i]);
                        put(1);
#pragma unroll
                        for (int i = 0; i < 8; ++i) h[i] = round_e5m2(rest_e5m2(h[i]));
                        put(2);
                    }
                    fence_async_shared();
                    tc_fence_before();
                    mbar_arrive(&sh.p_full);
                }
                // ---- the item's end: the next one's queries, then this one's output
                const AttnItem done = it;
                const int64_t end = it.u0 + it.ntiles;
                u = end;
                if (end < uend) {
                    next_item(p, it, items, rtiles);
                    prepare(sh.rows[item & 1 ^ 1]);
                }
                reduce_rows<RT>(l, [](float a, float b) { return a + b; });
                if (RT == 32 || (lane & 1) == 0) sh.top[wq][RT == 32 ? lane : lane >> 1] = l[0];
                // the shared part's results are there, and its partial results done with
                // (no wait but after a shared pass, whose end this kernel's start overlaps)
                if (item == 0) pdl_wait_primary();
                // the item's parts: this one alone, or [c0, c1]
                int c0 = part, c1 = part;
                if (done.u0 < part * share || end > part * share + share) {
                    c0 = (int)(done.u0 / share);
                    c1 = (int)((end - 1) / share);
                }
                bar_sync(bar, GT);
                float s = 0.0f, m = -INFINITY, back = 1.0f;  // of row `key`: sum, reference, what O is divided by
                if (key < RT) {
                    s = (sh.top[0][key] + sh.top[1][key]) + (sh.top[2][key] + sh.top[3][key]);
                    if (s > 0.0f || s != s) m = sh.ref[key];  // a NaN sum stays NaN
                    sh.fa[key] = back = 1.0f / sh.gain[key];  // (powers of two)
                }
                if (ok) ok = attn_wait(&sh.pv_done, (unsigned)((n - 1) & 1));
                tc_fence_after();
                bool write = true;
                if (c0 != c1) {
                    // Part c's results: slot 0 of a part holds the item that began before it, slot
                    // 1 the one that goes on after it.  The part that arrives last joins them, into
                    // its own O, and leaves the counter zero.
                    const int64_t slot = (int64_t)RT * (p.D + 2);
                    auto part_of = [&](int c) { return p.part + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * slot; };
                    float *mine = part_of(part);
                    bar_sync(bar, GT);
                    if (key < RT) {
                        __stcg(mine + (int64_t)RT * p.D + key, m);
                        __stcg(mine + (int64_t)RT * p.D + RT + key, s);
                    }
#pragma unroll
                    for (int h = 0; h < RT; h += 8) {
                        float o[kParts][8];
#pragma unroll
                        for (int c = 0; c < kParts; ++c) tc_ld8(o[c], to + c * RT + h);
                        tc_wait_ld();
                        if (key < p.D)
#pragma unroll
                            for (int r = 0; r < 8; ++r) __stcg(mine + (int64_t)(h + r) * p.D + key, (o[0][r] + o[1][r] + o[2][r]) * sh.fa[h + r]);
                    }
                    bar_sync(bar, GT);
                    if (key == 0) {  // (its fence covers what the barrier has shown it)
                        __threadfence();
                        sh.last = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
                        __threadfence();
                        if (sh.last) p.counters[c0] = 0u;
                    }
                    bar_sync(bar, GT);
                    write = sh.last;
                    if (write) {
                        // m = max m_c, l = sum l_c 2^(m_c - m), o = sum o_c 2^(m_c - m)
                        constexpr int TR = GT / RT;  // threads of a row; parts at a time
                        const int r = key / TR, k = key % TR, np = c1 - c0 + 1;
                        auto of_row = [&](int c) { return part_of(c0 + c) + (int64_t)RT * p.D + r; };
                        float mc = k < np ? __ldcg(of_row(k)) : -INFINITY, lc = k < np ? __ldcg(of_row(k) + RT) : 0.0f, mm = mc;
                        for (int c = k + TR; c < np; c += TR) mm = fmaxf(mm, __ldcg(of_row(c)));
#pragma unroll
                        for (int o = TR / 2; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(kFull, mm, o));
                        float ll = 0.0f;
#pragma unroll 1
                        for (int c = 0; c < np; c += TR) {
                            if (c > 0) {
                                mc = c + k < np ? __ldcg(of_row(c + k)) : -INFINITY;
                                lc = c + k < np ? __ldcg(of_row(c + k) + RT) : 0.0f;
                                bar_sync(bar, GT);
                            }
                            const float f = rel_weight(mc, mm);
                            ll += lc * f;
                            (&sh.top[0][0])[k * RT + r] = f;  // (TR * RT of them)
                            bar_sync(bar, GT);
                            const int some = min(TR, np - c);
#pragma unroll 1
                            for (int h = 0; h < RT; h += 16) {
                                float o[16];
                                if (c > 0) {
                                    tc_ld16(o, to + h);
                                    tc_wait_ld();
                                } else {
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = 0.0f;
                                }
#pragma unroll 2
                                for (int i = 0; i < some; ++i) {
                                    const float *q = part_of(c0 + c + i) + (int64_t)h * p.D + key, *g = &sh.top[0][0] + i * RT + h;
                                    float x[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) x[e] = key < p.D ? __ldcg(q + (int64_t)e * p.D) : 0.0f;
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        if (g[e] != 0.0f) o[e] = fmaf(x[e], g[e], o[e]);
                                }
                                tc_st16(to + h, reinterpret_cast<const uint32_t *>(o));
                            }
                        }
#pragma unroll
                        for (int o = TR / 2; o > 0; o >>= 1) ll += __shfl_xor_sync(kFull, ll, o);
#pragma unroll 1
                        for (int h = RT; h < kParts * RT; h += 16) {
                            uint32_t z[16] = {};
                            tc_st16(to + h, z);
                        }
                        bar_sync(bar, GT);  // (the weights are done with)
                        if (k == 0) {
                            sh.top[0][r] = mm;
                            sh.top[1][r] = ll;
                        }
                        bar_sync(bar, GT);
                        tc_wait_st();
                        if (key < RT) {
                            m = sh.top[0][key];
                            s = sh.top[1][key];
                            back = 1.0f;
                        }
                    }
                }
                if (write) {
                    if (key < RT) {
                        const int64_t row = w.out[key];
                        float fa = 0.0f, fc = 0.0f;
                        if (row >= 0) {
                            float lse2 = s > 0.0f || s != s ? m + lg2f(s) : -INFINITY;
                            fa = back;
                            if (p.mode == 0 && p.P > 0 && done.keys.ok) {
                                const float lp = p.pre_lse[row], mm = fmaxf(m, lp), a = rel_weight(m, mm), c = lp != lp ? lp : rel_weight(lp, mm);
                                s = s * a + c;
                                lse2 = s > 0.0f || s != s ? mm + lg2f(s) : -INFINITY;
                                fa *= a;
                                fc = c;
                            }
                            const float inv = lse2 == -INFINITY ? 0.0f : 1.0f / s;
                            fa *= inv;
                            fc *= inv;
                            if (p.mode == 1) p.pre_lse[row] = lse2;
                            else if (p.lse) p.lse[row] = lse2 * kLn2;
                        }
                        sh.fa[key] = fa;
                        sh.fc[key] = fc;
                    }
                    bar_sync(bar, GT);
                    const bool join = p.mode == 0 && p.P > 0 && done.keys.ok;
                    // (code that runs once an item stays short: it comes from far away)
#pragma unroll 1
                    for (int h = 0; h < RT; h += 8) {
                        float o[kParts][8], sp[8];
#pragma unroll
                        for (int c = 0; c < kParts; ++c) tc_ld8(o[c], to + c * RT + h);
#pragma unroll
                        for (int r = 0; r < 8; ++r) sp[r] = join && w.out[h + r] >= 0 && key < p.D ? p.pre_o[w.out[h + r] * p.D + key] : 0.0f;
                        tc_wait_ld();
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const int64_t row = w.out[h + r], at = row * p.D + key;
                            const float f = sh.fa[h + r];
                            float x = f == 0.0f ? 0.0f : (o[0][r] + o[1][r] + o[2][r]) * f;
                            if (join) x = fmaf(sp[r], sh.fc[h + r], x);
                            if (row >= 0 && key < p.D) {
                                if (p.mode == 1) p.pre_o[at] = x;
                                else static_cast<T *>(p.out)[at] = __float2bfloat16(x);
                            }
                        }
                    }
                }
                tc_fence_before();
                if (u >= uend) break;
                bar_sync(bar, GT);  // (the references and factors are done with)
                start_rows();
                bar_sync(bar, GT);
                ++item;
            }
        }
    }
    if (!ok && lane == 0) atomicOr(p.status, SPEC_FLAG_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == NW) tc_dealloc(tmem);
}

// ---- host ------------------------------------------------------------------
template <int NH, int RT, bool PLAIN> cudaError_t launch(const AttnParams &p, const CUtensorMap &cm, int sms, cudaStream_t s) {
    constexpr int smem = (int)sizeof(Tc8Smem<NH, RT>) + 1024;
    static_assert(smem <= 227 * 1024 && smem > 114 * 1024, "one block an SM: it takes all of TMEM");
    static_assert(kTeams * RT <= kAttnSlotRows && kTeams * kAttnSmsMax <= kAttnBlocksMax, "partial results of the teams");
    cudaError_t e = cudaFuncSetAttribute(attn8_tc_kernel<NH, RT, PLAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms < kAttnSmsMax ? sms : kAttnSmsMax));
    cfg.blockDim = dim3(128 * kTeams + 128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = p.mode == 0 && p.P > 0 ? 1 : 0;  // after the shared pass
    return cudaLaunchKernelEx(&cfg, attn8_tc_kernel<NH, RT, PLAIN>, p, cm);
}

template <int NH> cudaError_t launch_nh(const AttnParams &p, const CUtensorMap &cm, int sms, cudaStream_t s) {
    const int64_t rows = p.mode == 1 ? (int64_t)p.B * p.S * p.G : (int64_t)p.S * p.G;
    const bool plain = p.score.cap == 0.0f && !p.score.bias;
    if (plain) return rows <= 16 ? launch<NH, 16, true>(p, cm, sms, s) : launch<NH, 32, true>(p, cm, sms, s);
    return rows <= 16 ? launch<NH, 16, false>(p, cm, sms, s) : launch<NH, 32, false>(p, cm, sms, s);
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
