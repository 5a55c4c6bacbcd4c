// Attention over the 8-bit paged cache for bf16 queries on the fifth-generation
// tensor cores (attention.cuh: score, split, join; kv8.cuh: the cache's numbers).
//
// One persistent block per SM, in teams that know nothing of each other: a team has a
// warp that copies, 128 softmax threads for each 16 of an item's rows and its own
// share of the line of tiles (one warp issues the MMAs of all), so that what one waits
// for (a product's end, an item's first keys, its output) the others' work covers:
// three teams for up to 16 rows a cached head (group of queries x candidates), two of
// 32 rows, which share a tile's copies between two halves, for more.  A tile is 128
// keys, down the MMA's rows; the queries are its columns: a thread has a key, with
// the key's power of two, position and masks, and the MMA does no work for queries
// that are not there.  K and V go to the tensor cores as the codes they are:
//   * S^T = K Q^T.  A query, scaled by a power of two, is the sum of two e4m3 numbers
//     (8 significant bits, as bf16 has; the smallest elements may lose 2^-17 of the
//     largest); both products go into one accumulator.  A key's power of two
//     multiplies its scores.
//   * O^T = V^T P^T.  A weight of 2^-20 next to one of 1 is worth keeping where there are
//     many, and e4m3 ends at 2^-9.  So a weight times its key's power of two, relative
//     to the largest such product that the row has seen, is rounded to f16 and taken
//     apart into three e5m2 numbers: the upper byte of an f16 is one, and what it leaves
//     is an f16 again; the third is kept times 2^5.  So the parts cost an AND, a
//     subtraction and half a byte shuffle each, one multiplication in all, and hold 9
//     bits, or 2^-27 of the largest product: 2^20 keys that all end below it lose 2^-7
//     of that together.  (The largest power in its place, without the row's weight of it,
//     would let a V row that the row hardly sees, or a heavy one with little V, take the
//     others' bits.)  They are columns of one product and are added at the item's end.
//   * A row's largest score lies across the threads.  It is looked for, and the
//     largest product, in an item's first tile and where a score passes the reference
//     by 2^7 or a product its row's largest by 2^8, which one vote of the half's threads
//     finds (a thread compares its key's largest score with the smallest of the rows'
//     limits first); otherwise nobody needs another's scores.  Tiles go from the
//     last, which is full, to the first: with a bias by distance the largest scores
//     come first.  Sums of weights stay in the threads until the item's end.
//   * Where a tile hides keys, the threads look whether V holds NaN's code: such a row
//     becomes zeros and gives its NaN to the rows that see it; the rows that it is
//     hidden from see nothing.
//   * Pages that are a multiple of 8 entries come in boxes of the copy engine; of others
//     each lane copies 16 bytes of a row at a time: 64 x 5 queries on 2,048 entries in pages
//     of 5 280 us instead of 89 (CUDA cores: 664), single queries 1,329 instead of 377 (2,733).
//     That form is built once, for any scores.
//
// What bounds it.  Single queries on up to 32,768 entries, 64 requests, 8 heads of 128:
// 377 to 392 us by the GPU, up to 5.9 TB/s of the 6.65 that a copy reaches.  64 requests of
// 5 queries x group 4 on 2,048 entries: 89 us (3.1 TB/s; the tiles themselves run at 6.2):
// a team's start (13 us) and each change of items (some 12 us: the next queries, partial
// results, the first tile's references) run code that is in no cache any more and comes
// from far away, one miss of some 1,000 clk after another.  That is why the rest is short:
// 16 rows a thread (32, with the loops twice as long: 8 x 5 queries on 40 entries 15.1 us
// instead of 13, a shared prefix of 4,096 entries 137 instead of 130), one place for the
// queries of an item, the first or a later one (chain 91 -> 88 us, tree 324 -> 312), and why
// K and V ask L2 to let go of them first (single queries 406 -> 388 us, the chain 92 -> 89).
// 128 x 13 queries x group 4 on 2,048 entries, capped and biased, 325 us: bound by the
// softmax's instructions (30 a weight; half of the issue slots; the two halves' forms have 96
// registers, which spills some 80 bytes, because there are 19 warps) and the second reading of
// keys for the rows past 32; one tile of 64 rows, its threads at 96 registers, was no faster.
//
// The MMAs: an MMA of 128 x N x 32 takes 32 + N/4 clk, and 54 at least if its thread is
// not an elected one (the operands are then moved to uniform registers each time).
// Larger pages come in larger boxes: single queries on pages of 64 entries 360 to
// 379 us, of 128 354 to 378.
#include <cuda_fp16.h>

#include "attention.cuh"
#include "attn_tc.cuh"
#include "kv8.cuh"
#include "tma.cuh"

#include <type_traits>

namespace specv {
namespace {

constexpr int KT = 128, RT = 16, GT = 128;  // keys of a tile; rows that a thread has; threads that hold a tile's keys
constexpr int NT = 256;               // threads that plan
constexpr uint32_t kTile = KT * 128;  // bytes of 128 keys x up to 128 codes
constexpr int kInfo = 4;              // tiles whose notes are kept
constexpr float kNone = -1e30f;       // the reference of a row that has seen no key
constexpr float kLag = 7.0f;          // log2 of what a weight may reach
constexpr int kPowMin = 16;           // exponent byte that smaller products are taken relative to
constexpr int kUp = 7;                // log2 of a row's largest product of weight and power, when it was last looked for,
constexpr int kMore = 8;              // and how far it may grow until it is again: 2^(kUp + kMore) is an e5m2 number
constexpr int kLast = 5;              // log2 of what the last part is multiplied by (it is below 2^10)
constexpr int kParts = 3;             // e5m2 numbers that hold a weight
constexpr int kIdlePolls = 1 << 27;   // of the MMA warp without a product to issue: a poll takes tens of clk and,
                                      // unlike the other waits' tries, does not suspend, so this is seconds

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
// L2's policy for a copy: read once, or kept as anything else is
__device__ __forceinline__ uint64_t l2_policy(bool once) {
    uint64_t a, b;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(a));
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(b));
    return once ? a : b;
}
__device__ __forceinline__ void tma3_hint(uint32_t dst, const CUtensorMap *m, int x, int y, int z, unsigned long long *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(
            dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
// 16 bytes, or zeros where `bytes` is 0; a barrier's arrival when this thread's copies are there
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(unsigned long long *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// one of a warp's threads; the compiler knows that it is one
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0u;
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
__device__ __forceinline__ uint32_t last_e5m2(uint32_t h) {  // times 2^kLast
    const uint32_t up = (15u + kLast) << 10 | (15u + kLast) << 26;
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&up));
    uint16_t c;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t *>(&r)));
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

// What 16 of an item's rows have, for the 128 threads that hold a tile's keys.
struct Rows8 {
    alignas(16) float nref[RT], zero[RT];            // the references (log2 units), negated; zeros
    alignas(16) float corr[RT], corr_o[RT], gain[RT];  // what sums and O are multiplied by (at the
                                                     // end: O and the shared part); what weights are at a power of 1
    alignas(16) float most[RT], limit[RT];           // log2 of the largest product so far, to the reference (a weight of 1
                                                     // at a power of 1: 127); of the largest that fits
    alignas(16) float top[4][RT];                    // the warps' largest scores; at the end sums of weights
    alignas(16) float prod[4][RT];                   // and products, to those scores
    alignas(16) float join[GT / RT][RT];             // at a join: weights of some parts (a thread has a part and a row)
    alignas(16) float cf[RT];                        // what a product is multiplied by for log2 units or the cap's exponent
    alignas(16) float qp[RT], slope[RT];             // positions after the first; bias by distance, log2 units
    alignas(16) int low[RT];                         // first visible position
    AttnRows<RT> rows[2];
    unsigned words[RT][5];                           // a tile's candidates in the rows' tree masks
    float limit_min;                                 // the smallest of `limit`
    int qp0;                                         // the first position
    int low_max[2];                                  // the largest `low`, by turns of items
    int last;
};
// What a team has: HV times RT rows, 128 threads for each RT.
template <int NH, int HV> struct Team8 {
    static constexpr int kTeams = HV == 1 ? 3 : 2, kRows = HV * RT, kThreads = HV * GT;
    static constexpr int kSoftWarps = kTeams * HV * 4;
    static constexpr uint32_t kQ = kRows * 128;      // bytes of a part of the queries
    // P^T: 16 rows: a key's 64 bytes, three parts of four; 32: 32 bytes of a part, a part
    // after another
    static constexpr uint32_t kPart = KT * 32, kP = HV == 1 ? KT * 64 : kParts * kPart, kStep = HV == 1 ? 32 * 64 : 32 * 32;
    static constexpr int KS = 2;                     // buffers for K
    alignas(1024) unsigned char k[KS][kTile];
    alignas(1024) unsigned char v[kTile];
    alignas(1024) unsigned char q[2][kQ];            // the queries' first and second parts
    alignas(1024) unsigned char p[kP];
    Rows8 half[HV];
    unsigned sc[kInfo][2][KT / 4];                   // exponent bytes of a tile's K and V
    unsigned char bad[kInfo][KT / 4];                // a tile's keys with a bad block, four a byte
    int any_bad[kInfo];                              // whether there are any
    int first[kInfo];                                // whether an item begins
    alignas(8) unsigned long long k_full[KS], k_empty[KS], v_full, s_full[2], p_full, pv_done, q_full;
};
template <int NH, int HV> struct Tc8Smem {
    Team8<NH, HV> team[Team8<NH, HV>::kTeams];
    AttnPlan plan;
    uint32_t tmem;
};

__device__ __forceinline__ float sum_parts(const float (&o)[kParts][8], int r) {
    return fmaf(o[2][r], 1.0f / (1 << kLast), o[0][r] + o[1][r]);
}

// the item after `it` (one copy of this code)
static __device__ __noinline__ void next_item(const AttnParams &p, AttnItem &it, int items, int rtiles) {
    it = attn_next(p, it, items, rtiles, KT);
}
// The first key of an item's line of tiles: the last tile is full, the first has what
// is left (whole boxes).
__device__ __forceinline__ int line_start(const KeyLine &line, int ntiles) { return line.lo - (ntiles * KT - line.entries); }

template <int NH, int HV> constexpr int threads_of() {
    using H = Team8<NH, HV>;
    return 32 * (H::kSoftWarps + H::kTeams + 1);
}
// boxes: a page's rows come in boxes; else each lane copies 16 bytes of a row at a time
template <int NH, int HV, bool plain, bool boxes>
__global__ void __launch_bounds__((threads_of<NH, HV>()), 1)
    attn8_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap cache_map) {
    using H = Team8<NH, HV>;
    constexpr int G = H::kTeams, NW = H::kSoftWarps;  // teams; softmax warps
    using T = __nv_bfloat16;
    extern __shared__ unsigned char raw_[];
    Tc8Smem<NH, HV> &all = *reinterpret_cast<Tc8Smem<NH, HV> *>(
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw_) + 1023) & ~uintptr_t(1023)));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = warp < NW ? warp / (4 * HV) : warp < NW + G ? warp - NW : 0;  // then a warp a team for copies, one for MMAs
    H &sh = all.team[grp];
    const int per = p.S * p.G;
    const int64_t nrows = p.mode == 1 ? (int64_t)p.B * per : per;
    const int rtiles = (int)((nrows + H::kRows - 1) / H::kRows), items = p.H * rtiles;
    if (tid < G) {
        H &h = all.team[tid];
        for (int s = 0; s < H::KS; ++s) {
            mbar_init(&h.k_full[s], boxes ? 1 : 33);  // (rows: 32 lanes' copies, and the notes)
            mbar_init(&h.k_empty[s], 1);
        }
        mbar_init(&h.v_full, boxes ? 1 : 32);
        mbar_init(&h.s_full[0], 1);
        mbar_init(&h.s_full[1], 1);
        mbar_init(&h.p_full, H::kThreads);
        mbar_init(&h.pv_done, 1);
        mbar_init(&h.q_full, H::kThreads);
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
    constexpr uint32_t kO = 2 * G * H::kRows, kOCols = kParts * H::kRows;
    static_assert(kO + G * kOCols <= 512, "columns");
    bool ok = true;  // after a wait has run out nothing waits any more; the call is flagged
    if (warp == NW + G) {
        // ---------------- MMAs ----------------
        // A team's next product where its weights and V are there, its next scores where its
        // K is, and, of an item's first, the queries.
        if (elect_one()) {
            // Operands.  Scores: atoms of 8 rows x 128 bytes, the next 8 rows 1,024 bytes on;
            // 32 columns of K and Q are 32 bytes.  Values: the rows are keys, the products' K,
            // whose elements (V's columns: M; P's weights: N) are contiguous: 128 of V (zeros
            // past the head), 48 of P, or 32 and the next 32 a part further on.
            constexpr uint32_t id_s = tc_idesc8(H::kRows), id_o = tc_idesc_mn(kParts * H::kRows);
            int left = 0, idle = 0;
            int scored[G], weighed[G], begun[G], tiles[G];  // of the teams: tiles so far, items begun, tiles in all
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int64_t at = ((int64_t)g * gridDim.x + blockIdx.x) * share;
                scored[g] = weighed[g] = begun[g] = 0;
                left += tiles[g] = (int)max((int64_t)0, min(all.plan.total, at + share) - at);
            }
            while (left > 0 && idle < kIdlePolls) {
                ++idle;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    H &t = all.team[g];
                    const int n = scored[g], j = weighed[g];
                    if (j < n && mbar_test(&t.v_full, (unsigned)(j & 1)) && mbar_test(&t.p_full, (unsigned)(j & 1))) {
                        tc_fence_after();
                        if (!boxes) fence_async_shared();  // (the copies are ordinary writes)
                        const uint64_t a = tc_desc(smem_u32(t.v), 0, 1024),
                                       b = HV == 1 ? tc_desc64(smem_u32(t.p), 512) : tc_desc32(smem_u32(t.p), H::kPart, 256);
                        const uint32_t add = !t.first[j % kInfo];
#pragma unroll
                        for (int k = 0; k < KT / 32; ++k)
                            tc_mma8(tmem + kO + g * kOCols, a + k * (4096 / 16), b + k * (H::kStep / 16), id_o, k > 0 ? 1u : add);
                        tc_commit(&t.pv_done);
                        weighed[g] = j + 1;
                        --left;
                        idle = 0;
                    }
                    if (n < tiles[g] && n < weighed[g] + 2 && mbar_test(&t.k_full[n % H::KS], (unsigned)((n / H::KS) & 1))) {
                        const bool first = t.first[n % kInfo];
                        if (!first || mbar_test(&t.q_full, (unsigned)(begun[g] & 1))) {
                            tc_fence_after();
                            if (!boxes) fence_async_shared();
                            const uint64_t a = tc_desc(smem_u32(t.k[n % H::KS]), 16, 1024), b = tc_desc(smem_u32(t.q[0]), 16, 1024);
#pragma unroll
                            for (int k = 0; k < NH * 4; ++k)  // first parts, second parts
                                tc_mma8(tmem + (2 * g + (n & 1)) * H::kRows, a + (k % (NH * 2)) * (32 / 16),
                                        b + (k / (NH * 2)) * (H::kQ / 16) + (k % (NH * 2)) * (32 / 16), id_s, k > 0);
                            tc_commit(&t.k_empty[n % H::KS]);
                            tc_commit(&t.s_full[n & 1]);
                            scored[g] = n + 1;
                            begun[g] += first;
                            idle = 0;
                        }
                    }
                }
            }
            ok = left == 0;
        }
        ok = __all_sync(kFull, ok);  // (any lane may have been elected; lane 0 reports)
    } else if (u < uend) {
        AttnItem it = attn_find<NT>(p, all.plan, u, items, rtiles, KT);
        if (warp >= NW) {
            // ---------------- copies ----------------
            // A shared prefix is read by many; the others' keys, once, would push the code that
            // runs once an item out of L2.
            const uint64_t policy = l2_policy(p.mode == 0);
            const int nbox = boxes ? KT / p.box : 0;
            const int zero_row = (int)(2 * p.nb * p.bs);  // past the map: zeros are written
            const int v_row = (int)(p.nb * p.bs);
            const bool four = boxes || p.box == 4;              // four neighbours lie in one page
            const int chunk = lane & 7, mine = lane >> 3; // a lane's 16 bytes of four rows
            const uint32_t to0 = mine * 128 + ((chunk ^ mine) << 4), to1 = (4 + mine) * 128 + ((chunk ^ (4 + mine)) << 4);
            const int64_t stride = (int64_t)p.H * p.D;
            int n = 0;
            while (true) {
                if (!it.keys.ok && u == it.u0 && it.h == 0 && it.rt == 0 && lane == 0) attn_flag(p, it.b);
                const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
                const int *table = p.mode == 1 ? p.stable : p.table + (int64_t)it.b * p.max_blocks;
                const KeyLine line = it.keys.ok ? attn_line(p, it.keys) : KeyLine{0, 0};
                // A lane looks up 4 keys: their blocks (in whole boxes, or fours, the first's)
                // two tiles ahead, their exponents one; a box's row comes from the lane that
                // has its first key.
                int blk[4] = {0, 0, 0, 0}, row[4] = {};
                unsigned ks = 0u, vs = 0u, bad = 0u;
                const int start = line_start(line, it.ntiles);
                auto has = [&](int t, int e) {
                    const int c = start + t * KT + lane * 4 + e;
                    return t >= t0 && it.keys.ok && c >= line.lo && c < it.keys.hi;
                };
                auto blocks_of = [&](int t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e == 0 || !four)
                            blk[e] = has(t, e) ? __ldg(table + fast_div((unsigned)(start + t * KT + lane * 4 + e), p.bs_div)) : 0;
                };
                auto entries_of = [&](int t) {
                    ks = vs = bad = 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (e > 0 && four) break;
                        row[e] = zero_row;
                        if (!has(t, e)) continue;
                        const int c = start + t * KT + lane * 4 + e, at = c - (int)fast_div((unsigned)c, p.bs_div) * p.bs;
                        if (blk[e] < 0 || (int64_t)blk[e] >= p.nb) {
                            bad |= (four ? 0xfu : 1u) << e;
                            continue;
                        }
                        row[e] = blk[e] * p.bs + at;
                        const int64_t s = ((int64_t)blk[e] * p.H + it.h) * p.bs + at;
                        if (four) {
                            ks = __ldg(reinterpret_cast<const unsigned *>(p.ks + s));
                            vs = __ldg(reinterpret_cast<const unsigned *>(p.vs + s));
                        } else {
                            ks |= (unsigned)__ldg(p.ks + s) << (8 * e);
                            vs |= (unsigned)__ldg(p.vs + s) << (8 * e);
                        }
                    }
                };
                // rows r of a plane (0: K, v_row: V), zeros where there is none
                auto copy = [&](unsigned char *to, unsigned long long *bar, const int (&r)[4], int plane) {
                    const uint32_t dst = smem_u32(to);
                    if (boxes) {
                        const int x = __shfl_sync(kFull, r[0], lane < nbox ? lane * p.box >> 2 : 0);
                        if (lane == 0) mbar_arrive_expect_tx(bar, kTile);
                        __syncwarp();
                        if (lane < nbox)
                            tma3_hint(dst + (uint32_t)(lane * p.box) * 128u, &cache_map, 0, it.h, x == zero_row ? x : x + plane, bar, policy);
                        return;
                    }
                    const unsigned char *src = static_cast<const unsigned char *>(plane ? p.vc : p.kc) + (int64_t)it.h * p.D + chunk * 16;
#pragma unroll 8
                    for (int i = 0; i < 32; ++i) {
                        int x = __shfl_sync(kFull, r[0], i);
                        if (!four) {
                            const int b = __shfl_sync(kFull, r[1], i), c = __shfl_sync(kFull, r[2], i), d = __shfl_sync(kFull, r[3], i);
                            x = mine == 0 ? x : mine == 1 ? b : mine == 2 ? c : d;
                        } else if (x != zero_row) {
                            x += mine;
                        }
                        const bool is = x != zero_row && chunk * 16 < p.D;
                        cp_async16(dst + (i >> 1) * 1024 + (i & 1 ? to1 : to0), is ? src + x * stride : p.kc, is ? 16 : 0);
                    }
                    cp_async_arrive(bar);
                };
                blocks_of(t1 - 1);
                entries_of(t1 - 1);
                blocks_of(t1 - 2);
                int row_v[4] = {zero_row, zero_row, zero_row, zero_row};
                // the order of use: K0 K1 V0 K2 V1 ...
#pragma unroll 1
                for (int t = t1 - 1; t >= t0 - 1; --t) {
                    int before[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) before[e] = row_v[e];
                    if (t >= t0) {
                        if (bad) attn_flag(p, it.b);
                        const int i = n % kInfo, s = n % H::KS;
                        const bool any = __any_sync(kFull, bad != 0u);
                        if (n >= H::KS && ok) ok = attn_wait(&sh.k_empty[s], (unsigned)((n / H::KS - 1) & 1));
                        sh.sc[i][0][lane] = ks;
                        sh.sc[i][1][lane] = vs;
                        sh.bad[i][lane] = (unsigned char)bad;
                        if (lane == 0) {
                            sh.any_bad[i] = any;
                            sh.first[i] = t == t1 - 1;
                        }
                        // the notes, before an arrival that releases them (a lane's copies
                        // arrive on their own and release no other writes)
                        __syncwarp();
                        if (!boxes && lane == 0) mbar_arrive(&sh.k_full[s]);
                        copy(sh.k[s], &sh.k_full[s], row, 0);
#pragma unroll
                        for (int e = 0; e < 4; ++e) row_v[e] = row[e];
                        entries_of(t - 1);
                        blocks_of(t - 2);
                        ++n;
                    }
                    if (t < t1 - 1) {
                        const int j = n - (t >= t0 ? 2 : 1);
                        if (j > 0 && ok) ok = attn_wait(&sh.pv_done, (unsigned)((j - 1) & 1));
                        __syncwarp();
                        copy(sh.v, &sh.v_full, before, v_row);
                    }
                }
                u = it.u0 + it.ntiles;
                if (u >= uend) break;
                next_item(p, it, items, rtiles);
            }
            // no copy may land after the block has gone
            if (!boxes) asm volatile("cp.async.wait_all;" ::: "memory");
            for (int i = max(0, n - H::KS); i < n; ++i) ok = mbar_drain(&sh.k_full[i % H::KS], (unsigned)((i / H::KS) & 1)) && ok;
            ok = mbar_drain(&sh.v_full, (unsigned)((n - 1) & 1)) && ok;
        } else {
            // ---------------- softmax ----------------
            const int wq = warp & 3, key = tid & (GT - 1);            // key of a tile; row of the MMA: TMEM lane
            const int half = HV == 1 ? 0 : (warp >> 2) & 1;            // of the item's rows
            const int bar = 2 + (warp >> 2);                          // the half's barrier; the team's
            auto team_sync = [&] { bar_sync(HV == 1 ? bar : 2 + NW / 4 + grp, H::kThreads); };
            Rows8 &hs = sh.half[half];
            const uint32_t lanes = (uint32_t)(wq * 32) << 16;
            const uint32_t col_s = tmem + grp * 2 * H::kRows + half * RT + lanes, to = tmem + kO + grp * kOCols + half * RT + lanes;
            const bool by_pos = p.window > 0 || p.first != nullptr;
            const uint32_t neg = p.score.scale < 0.0f ? 0x80008000u : 0u;  // a negative scale: the queries are negated
            const bool cap = !plain && p.score.cap > 0.0f;
            // Scores are log2 units; capped ones (cap_score) without the cap itself, which
            // all have in common: lse gets it back.
            const float scale = fabsf(p.score.scale) * (cap ? p.score.cap_arg : kLog2e);
            const float2 cap2 = pair(-2.0f * kLog2e * p.score.cap, -2.0f * kLog2e * p.score.cap);
            const float shift = cap ? kLog2e * p.score.cap : 0.0f;
            constexpr unsigned kRowLanes = 0xffffu;
            int item = 0, n = 0;
            auto start_rows = [&] {  // of an item: nothing seen yet
                if (key < RT) {
                    hs.nref[key] = -kNone;
                    hs.zero[key] = 0.0f;
                    hs.most[key] = kNone;
                    hs.gain[key] = pow2i(127 + kUp - kPowMin);
                }
            };
            // An item's rows and queries: 8 elements a thread at a time.
            auto prepare = [&](int turn) {
                AttnRows<RT> &w = hs.rows[turn];
                AttnItem of = it;
                of.rt = it.rt * HV + half;
                attn_rows<RT, GT>(p, of, w, key);
                if (key < RT) {
                    const int lo = max(w.first[key], p.window > 0 ? w.qp[key] - p.window + 1 : (int)0x80000000);
                    hs.low[key] = lo;
                    const bool is = w.out[key] >= 0;
                    const int most = __reduce_max_sync(kRowLanes, is ? lo : (int)0x80000000);
                    const int qp0 = __reduce_min_sync(kRowLanes, is ? w.qp[key] : 0x7fffffff);
                    hs.qp[key] = is ? (float)pos_dist(w.qp[key], qp0) : 0.0f;
                    hs.slope[key] = -kLog2e * w.slope[key];
                    if (lane == 0) {
                        hs.low_max[turn] = most;
                        hs.qp0 = qp0;
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
                    if (key % LR == 0) hs.cf[r] = scale * kv8_power(s);
                    uint32_t a[2], b[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        a[e] = kv8_code2(x[4 * e] * f, x[4 * e + 1] * f) | kv8_code2(x[4 * e + 2] * f, x[4 * e + 3] * f) << 16;
                        const float4 y = kv8_value4(a[e]);
                        b[e] = kv8_code2(x[4 * e] * f - y.x, x[4 * e + 1] * f - y.y) |
                               kv8_code2(x[4 * e + 2] * f - y.z, x[4 * e + 3] * f - y.w) << 16;
                    }
                    const uint32_t at = (half * RT + r) * 128 + (((d >> 4) ^ (r & 7)) << 4) + (d & 8);
                    *reinterpret_cast<uint2 *>(sh.q[0] + at) = make_uint2(a[0], a[1]);
                    *reinterpret_cast<uint2 *>(sh.q[1] + at) = make_uint2(b[0], b[1]);
                }
                fence_async_shared();
                team_sync();
                mbar_arrive(&sh.q_full);
            };
            // An item's turn: its queries, the output of the item before, its tiles.
            AttnItem done = it;
            float l[RT];                         // sums of this thread's weights
            for (bool more = true;; ++item) {
                if (more) prepare(item & 1);
                if (item > 0) {
                    const AttnRows<RT> &w = hs.rows[(item & 1) ^ 1];
                    reduce_rows<RT>(l, [](float a, float b) { return a + b; });
                    if ((lane & 1) == 0) hs.top[wq][lane >> 1] = l[0];
                    // the shared part's results are there, and its partial results done with
                    // (no wait but after a shared pass, whose end this kernel's start overlaps)
                    if (item == 1) pdl_wait_primary();
                    // the item's parts: this one alone, or [c0, c1]
                    int c0 = part, c1 = part;
                    if (done.u0 < part * share || done.u0 + done.ntiles > part * share + share) {
                        c0 = (int)(done.u0 / share);
                        c1 = (int)((done.u0 + done.ntiles - 1) / share);
                    }
                    bar_sync(bar, GT);
                    float s = 0.0f, m = -INFINITY, back = 1.0f;  // of row `key`: sum, reference, what O is divided by
                    if (key < RT) {
                        s = (hs.top[0][key] + hs.top[1][key]) + (hs.top[2][key] + hs.top[3][key]);
                        if (s > 0.0f || s != s) m = shift - hs.nref[key];  // a NaN sum stays NaN
                        hs.corr[key] = back = 1.0f / hs.gain[key];  // (powers of two)
                    }
                    if (ok) ok = attn_wait(&sh.pv_done, (unsigned)((n - 1) & 1));
                    tc_fence_after();
                    bool write = true;
                    if (c0 != c1) {
                        // Part c's results: slot 0 of a part holds the item that began before it, slot
                        // 1 the one that goes on after it.  The part that arrives last joins them, into
                        // its own O, and leaves the counter zero.
                        const int64_t slot = (int64_t)RT * (p.D + 2);
                        auto part_of = [&](int c) { return p.part + (((int64_t)c * 2 + (c == c0 ? 1 : 0)) * HV + half) * slot; };
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
                            for (int c = 0; c < kParts; ++c) tc_ld8(o[c], to + c * H::kRows + h);
                            tc_wait_ld();
                            if (key < p.D)
#pragma unroll
                                for (int r = 0; r < 8; ++r) __stcg(mine + (int64_t)(h + r) * p.D + key, sum_parts(o, r) * hs.corr[h + r]);
                        }
                        bar_sync(bar, GT);
                        if (key == 0) {  // (its fence covers what the barrier has shown it)
                            __threadfence();
                            hs.last = atomicAdd(p.counters + c0 * HV + half, 1u) == (unsigned)(c1 - c0);
                            __threadfence();
                            if (hs.last) p.counters[c0 * HV + half] = 0u;
                        }
                        bar_sync(bar, GT);
                        write = hs.last;
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
                                hs.join[k][r] = f;
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
                                        const float *q = part_of(c0 + c + i) + (int64_t)h * p.D + key, *g = &hs.join[i][h];
                                        float x[16];
#pragma unroll
                                        for (int e = 0; e < 16; ++e) x[e] = key < p.D ? __ldcg(q + (int64_t)e * p.D) : 0.0f;
#pragma unroll
                                        for (int e = 0; e < 16; ++e) o[e] = fmaf(x[e], g[e], o[e]);  // (a weight of 0 keeps V's NaN)
                                    }
                                    tc_st16(to + h, reinterpret_cast<const uint32_t *>(o));
                                }
                                tc_wait_st();  // (the next parts' sums begin with a load of these)
                            }
#pragma unroll
                            for (int o = TR / 2; o > 0; o >>= 1) ll += __shfl_xor_sync(kFull, ll, o);
#pragma unroll 1
                            for (int c = 1; c < kParts; ++c) {
                                uint32_t z[RT] = {};
                                tc_st16(to + c * H::kRows, z);
                            }
                            bar_sync(bar, GT);  // (the weights are done with)
                            if (k == 0) {
                                hs.top[0][r] = mm;
                                hs.top[1][r] = ll;
                            }
                            bar_sync(bar, GT);
                            tc_wait_st();
                            if (key < RT) {
                                m = hs.top[0][key];
                                s = hs.top[1][key];
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
                            hs.corr[key] = fa;
                            hs.corr_o[key] = fc;
                        }
                        bar_sync(bar, GT);
                        const bool join = p.mode == 0 && p.P > 0 && done.keys.ok;
                        // (code that runs once an item stays short: it comes from far away)
#pragma unroll 1
                        for (int h = 0; h < RT; h += 8) {
                            float o[kParts][8], sp[8];
#pragma unroll
                            for (int c = 0; c < kParts; ++c) tc_ld8(o[c], to + c * H::kRows + h);
#pragma unroll
                            for (int r = 0; r < 8; ++r) sp[r] = join && w.out[h + r] >= 0 && key < p.D ? p.pre_o[w.out[h + r] * p.D + key] : 0.0f;
                            tc_wait_ld();
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                const int64_t row = w.out[h + r], at = row * p.D + key;
                                const float f = hs.corr[h + r];
                                float x = sum_parts(o, r) * f;  // (a row that sees nothing: zeros; f = 0 keeps V's NaN)
                                if (join) x = fmaf(sp[r], hs.corr_o[h + r], x);
                                if (row >= 0 && key < p.D) {
                                    if (p.mode == 1) p.pre_o[at] = x;
                                    else static_cast<T *>(p.out)[at] = __float2bfloat16(x);
                                }
                            }
                        }
                    }
                    tc_fence_before();
                }
                if (!more) break;
                bar_sync(bar, GT);  // (the references and factors are done with)
                start_rows();
                bar_sync(bar, GT);
                const AttnRows<RT> &w = hs.rows[item & 1];
                const int t0 = (int)(u - it.u0), t1 = (int)(min(uend, it.u0 + it.ntiles) - it.u0);
                const KeyLine line = it.keys.ok ? attn_line(p, it.keys) : KeyLine{0, 0};
                const int start = line_start(line, it.ntiles);
                const int qp0 = hs.qp0;
                const int low_max = max(hs.low_max[item & 1], sh.half[HV - 1 - half].low_max[item & 1]);  // (every row's)
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
                    const int vs = sc[KT + key];
                    const float pw = vs == 255 ? 0.0f : (float)vs;
                    const int bad = sh.any_bad[n % kInfo];
                    // whether the tile may mask a key: the line's ends, candidates, a bad
                    // block, the window's and the document's first tile
                    const bool special = !it.keys.ok || c0 < it.keys.lo || c0 + KT > it.keys.len ||
                                         bad || (by_pos && (p.key_pos || c0 < low_max));
                    const int cand = c0 + key - it.keys.len;           // the key as a candidate, or < 0
                    bool in = true;
                    if (special) {
                        in = it.keys.ok && c0 + key >= it.keys.lo && c0 + key < it.keys.hi &&
                             !((sh.bad[n % kInfo][key >> 2] >> (key & 3)) & 1);
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
                                hs.words[r][i - r * 5] = x < p.W ? p.mask[((int64_t)it.b * p.S + w.cand[r]) * p.W + x] : 0u;
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
                                bool s = !by_pos || kp >= hs.low[r];
                                if (p.mode == 0 && cand >= 0) s = s && (tree ? (hs.words[r][x] >> (cand & 31)) & 1u : cand <= w.cand[r]);
                                seen |= (unsigned)s << r;
                            }
                        }
                    }
                    const uint32_t ts = col_s + (n & 1) * H::kRows;
                    const float kd = (float)pos_dist(qp0, kp);
                    const float2 kd2 = pair(kd, kd);
                    // Scores in log2 units less the references; without them (raw) to find new ones.
                    float y[RT];
                    bool raw = n == n0;
#pragma unroll 1
                    while (true) {
                        tc_ld16(y, ts);
                        tc_wait_ld();
                        const float2 kf2 = pair(kf, kf);
#pragma unroll
                        for (int r = 0; r < RT; r += 4) {  // (the key's factor first: with the query's it is the score's size)
                            const float2 a = __fmul2_rn(pair(y[r], y[r + 1]), kf2), b = __fmul2_rn(pair(y[r + 2], y[r + 3]), kf2);
                            y[r] = a.x, y[r + 1] = a.y, y[r + 2] = b.x, y[r + 3] = b.y;
                        }
                        const float *nref = raw ? hs.zero : hs.nref;
                        if (cap) {
                            const float2 one = pair(1.0f, 1.0f);
#pragma unroll
                            for (int r = 0; r < RT; r += 4) {
                                const float4 c = *reinterpret_cast<const float4 *>(&hs.cf[r]);
                                float2 a = __fmul2_rn(pair(y[r], y[r + 1]), pair(c.x, c.y)), b = __fmul2_rn(pair(y[r + 2], y[r + 3]), pair(c.z, c.w));
                                a = __fadd2_rn(pair(ex2f(a.x), ex2f(a.y)), one), b = __fadd2_rn(pair(ex2f(b.x), ex2f(b.y)), one);
                                y[r] = rcpf(a.x), y[r + 1] = rcpf(a.y), y[r + 2] = rcpf(b.x), y[r + 3] = rcpf(b.y);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < RT; r += 4) {
                            const float4 m = *reinterpret_cast<const float4 *>(nref + r);
                            float2 a = pair(m.x, m.y), b = pair(m.z, m.w), ca = cap2, cb = cap2;
                            if (!plain && p.score.bias) {  // (both terms of the distance are positive for entries: no cancellation)
                                const float4 q = *reinterpret_cast<const float4 *>(&hs.qp[r]), s = *reinterpret_cast<const float4 *>(&hs.slope[r]);
                                a = __ffma2_rn(pair(s.x, s.y), __fadd2_rn(pair(q.x, q.y), kd2), a);
                                b = __ffma2_rn(pair(s.z, s.w), __fadd2_rn(pair(q.z, q.w), kd2), b);
                            }
                            if (!cap) {
                                const float4 c = *reinterpret_cast<const float4 *>(&hs.cf[r]);
                                ca = pair(c.x, c.y), cb = pair(c.z, c.w);
                            }
                            a = __ffma2_rn(pair(y[r], y[r + 1]), ca, a), b = __ffma2_rn(pair(y[r + 2], y[r + 3]), cb, b);
                            y[r] = a.x, y[r + 1] = a.y, y[r + 2] = b.x, y[r + 3] = b.y;
                        }
                        if (special) {
#pragma unroll
                            for (int r = 0; r < RT; ++r) y[r] = (seen >> r) & 1u ? y[r] : -INFINITY;
                        }
                        if (!raw) {
                            float over = -INFINITY;
#pragma unroll
                            for (int r = 0; r < RT; r += 2) over = fmaxf(fmaxf(over, y[r]), y[r + 1]);
                            bool more = over > kLag;
                            if (over + pw > hs.limit_min) {  // perhaps a product: rows differ
#pragma unroll
                                for (int r = 0; r < RT; r += 4) {
                                    const float4 m = *reinterpret_cast<const float4 *>(&hs.limit[r]);
                                    more = more || y[r] + pw > m.x || y[r + 1] + pw > m.y || y[r + 2] + pw > m.z || y[r + 3] + pw > m.w;
                                }
                            }
                            if (!bar_or(bar, GT, more)) break;
                            raw = true;
                            continue;
                        }
                        // The tile's largest scores and products, these relative to the warp's largest
                        // score (so that they are exact, however far from zero scores are); a new
                        // reference where a row's score has grown past 2^kLag of the old one.
                        float mine = -INFINITY, prod = -INFINITY;  // of row `lane`
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const float m = warp_max(y[r]), g = warp_max(y[r] - m + pw);
                            if (lane == r) mine = m, prod = g;
                        }
                        if (lane < RT) {
                            hs.top[wq][lane] = mine;
                            hs.prod[wq][lane] = prod;
                        }
                        bar_sync(bar, GT);
                        if (key < RT) {
                            const float top = fmaxf(fmaxf(hs.top[0][key], hs.top[1][key]), fmaxf(hs.top[2][key], hs.top[3][key]));
                            const float old = -hs.nref[key];
                            const bool grew = top > old + kLag || (old == kNone && top > kNone);
                            const float ref = grew ? top : old, by = old - ref;
                            float most = hs.most[key] + by;
#pragma unroll
                            for (int i = 0; i < 4; ++i) most = fmaxf(most, hs.prod[i][key] + (hs.top[i][key] - ref));
                            // (a weight may be above 1: the gain's power of two stays a normal number)
                            const int was = 127 + kUp - ((int)(__float_as_uint(hs.gain[key]) >> 23) - 127);
                            const int now = min(max((int)ceilf(most), kPowMin), 254);
                            hs.most[key] = most;
                            hs.limit[key] = (float)(now + kMore);
                            hs.corr[key] = grew ? ex2f(by) : 1.0f;
                            hs.corr_o[key] = grew ? ex2f(by + (float)(was - now)) : pow2i(was - now);
                            hs.gain[key] = pow2i(127 + kUp - now);
                            if (grew) hs.nref[key] = -top;
                            // (rows that have seen nothing pass kLag at their first key)
                            const int least = __reduce_min_sync(kRowLanes, ref > kNone ? now + kMore : 254 + kMore);
                            if (lane == 0) hs.limit_min = (float)least;
                        }
                        bar_sync(bar, GT);
#pragma unroll
                        for (int r = 0; r < RT; r += 4) {
                            const float4 m = *reinterpret_cast<const float4 *>(&hs.nref[r]), f = *reinterpret_cast<const float4 *>(&hs.corr[r]);
                            y[r] += m.x, y[r + 1] += m.y, y[r + 2] += m.z, y[r + 3] += m.w;
                            l[r] *= f.x, l[r + 1] *= f.y, l[r + 2] *= f.z, l[r + 3] *= f.w;
                        }
                        if (n > n0) {  // O, still once the product before has ended
                            if (ok) ok = attn_wait(&sh.pv_done, (unsigned)((n - 1) & 1));
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < kParts; ++c) {
                                const uint32_t at = to + c * H::kRows;
                                float o[RT];
                                uint32_t z[RT];
                                tc_ld16(o, at);
                                tc_wait_ld();
#pragma unroll
                                for (int r = 0; r < RT; ++r) z[r] = __float_as_uint(o[r] * hs.corr_o[r]);
                                tc_st16(at, z);
                            }
                            tc_wait_st();
                        }
                        break;
                    }
                    bool nan_v = vs == 255;
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
                        if (HV > 1) team_sync();  // (both have looked)
                        if (nan & 0x80808080u) {
                            nan_v = true;
#pragma unroll 1
                            for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(vr + (i << 4)) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    // P's buffer is free once the product before has ended
                    if (n > n0 && ok) ok = attn_wait(&sh.pv_done, (unsigned)((n - 1) & 1));
                    // weights: summed, times V's power of two to three e5m2 numbers
                    unsigned char *pp = sh.p + key * (HV == 1 ? 64 : 32);
                    const int sw = HV == 1 ? (key >> 1) & 3 : (key >> 2) & 1;  // the swizzle of 64 or 32 bytes
                    const float vf = nan_v ? 0.0f : kv8_power(vs);
                    const float2 vf2 = pair(vf, vf);
                    {
                        uint32_t h[RT / 2];
#pragma unroll
                        for (int i = 0; i < RT / 2; ++i) {
                            const int q = 2 * i;
                            const float2 g = *reinterpret_cast<const float2 *>(&hs.gain[q]);
                            const float2 a = pair(ex2f(y[q]), ex2f(y[q + 1]));
                            const float2 sum = __fadd2_rn(pair(l[q], l[q + 1]), a);
                            l[q] = sum.x, l[q + 1] = sum.y;
                            // (the gain first: a hidden key's power may be any, its weight stays 0)
                            const float2 b = __fmul2_rn(__fmul2_rn(a, g), vf2);
                            h[i] = pack_f16(b.x, b.y);
                        }
                        auto put = [&](int c) {
                            uint32_t z[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) z[i] = c < 2 ? __byte_perm(h[2 * i], h[2 * i + 1], 0x7531) : h[2 * i] | h[2 * i + 1] << 16;
                            *reinterpret_cast<uint4 *>(pp + (HV == 1 ? (c ^ sw) << 4 : c * H::kPart + ((half ^ sw) << 4))) = make_uint4(z[0], z[1], z[2], z[3]);
                        };
                        put(0);
#pragma unroll
                        for (int i = 0; i < RT / 2; ++i) h[i] = rest_e5m2(h[i]);
                        put(1);
#pragma unroll
                        for (int i = 0; i < RT / 2; ++i) h[i] = last_e5m2(rest_e5m2(h[i]));
                        put(2);
                    }
                    if (nan_v) {  // the rows that see it get NaN, the others nothing
#pragma unroll 1
                        for (int r = 0; r < RT; ++r)
                            if ((seen >> r) & 1u)
                                pp[((half ^ sw) << 4) + r] = 0x7f;
                    }
                    fence_async_shared();
                    tc_fence_before();
                    mbar_arrive(&sh.p_full);
                }
                done = it;
                u = it.u0 + it.ntiles;
                more = u < uend;
                if (more) next_item(p, it, items, rtiles);
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
template <int NH, int HV, bool PLAIN, bool BOXES> cudaError_t launch(const AttnParams &p, const CUtensorMap &cm, int sms, cudaStream_t s) {
    constexpr int smem = (int)sizeof(Tc8Smem<NH, HV>) + 1024;
    static_assert(smem <= 227 * 1024 && smem > 114 * 1024, "one block an SM: it takes all of TMEM");
    using H = Team8<NH, HV>;
    static_assert(H::kTeams * H::kRows <= kAttnSlotRows && H::kTeams * HV * kAttnSmsMax <= kAttnBlocksMax, "partial results of the teams");
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = ensure_smem_attr(attn8_tc_kernel<NH, HV, PLAIN, BOXES>, smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms < kAttnSmsMax ? sms : kAttnSmsMax));
    cfg.blockDim = dim3((threads_of<NH, HV>()));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = p.mode == 0 && p.P > 0 ? 1 : 0;  // after the shared pass
    return cudaLaunchKernelEx(&cfg, attn8_tc_kernel<NH, HV, PLAIN, BOXES>, p, cm);
}

template <int NH> cudaError_t launch_nh(const AttnParams &p, const CUtensorMap &cm, int sms, cudaStream_t s) {
    const int64_t rows = p.mode == 1 ? (int64_t)p.B * p.S * p.G : (int64_t)p.S * p.G;
    const bool plain = p.score.cap == 0.0f && !p.score.bias;
    auto go = [&](auto hv) {
        constexpr int HV = decltype(hv)::value;
        if (p.box < 8) return launch<NH, HV, false, false>(p, cm, sms, s);
        return plain ? launch<NH, HV, true, true>(p, cm, sms, s) : launch<NH, HV, false, true>(p, cm, sms, s);
    };
    return rows <= RT ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 2>{});
}

}  // namespace

// Rows of a page a box takes, as attn_tc_box; of pages that are not whole boxes, or where
// exponents cannot be read four at a time: 4, or 1, rows whose look-up is shared.
int attn8_tc_box(const AttnParams &p) {
    if (p.D > 128 || 2 * p.nb * p.bs > 0x7fffff00LL) return 0;
    if (reinterpret_cast<uintptr_t>(p.ks) % 4 != 0 || p.bs % 4 != 0) return 1;
    const int box = attn_tc_box(p);
    return box ? box : 4;
}

cudaError_t launch_attn8_tc(const AttnParams &p, int sms, cudaStream_t s) {
    CUtensorMap cm = {};
    if (p.box >= 8) {
        const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.H, (cuuint64_t)(2 * p.nb * p.bs)};
        const cuuint64_t strides[2] = {(cuuint64_t)p.D, (cuuint64_t)p.H * p.D};
        const cuuint32_t box[3] = {128, 1, (cuuint32_t)p.box}, ones[3] = {1, 1, 1};
        if (tc_encode_fn()(&cm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(p.kc), dims, strides, box, ones,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    return p.D <= 64 ? launch_nh<1>(p, cm, sms, s) : launch_nh<2>(p, cm, sms, s);
}

}  // namespace specv
