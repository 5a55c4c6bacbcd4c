// Shared device code of the paged-cache attention kernels (sm_103a): the
// score, the split of the work over the grid, and the join of split results.
//
// Work.  A tile is `kt` consecutive keys; an item is a (request, cached head,
// row tile) with its keys in tiles, rows being the S * Hq/H queries that share
// the cached head.  The pass over a shared prefix is one request whose rows
// are every request's.  All items' tiles form one line; block i takes tiles
// [i*share, (i+1)*share), so lengths from one token to the longest give every
// block the same work.  An item that lies in several blocks leaves its partial
// results in the workspace, and they are joined in block order: by the block
// that arrives last, or by a second kernel (attn_join.cu), which costs a call
// that splits nothing 3 to 4 us but joins large items with all SMs.
#pragma once

#include "attn_params.h"
#include "common.cuh"
#include "tma.cuh"

namespace specv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The hardware's 2^x (2 ulp) and log2 (2^-22), in float32 calls for the joins and lse
// only: a partial sum's weight moves by 2^-22 of itself, lse by 2^-22, which its own
// rounding reaches from 4 on.  (The weights of a float32 call are exp2f's.)
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2f(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcpf(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// mbar_wait_bounded in a few instructions: the kernels wait in many places.
__device__ __forceinline__ bool attn_wait(unsigned long long *bar, unsigned phase) {
#pragma unroll 1
    for (int i = 0; i < (int)kSpinLimit; ++i)
        if (mbar_try_wait(bar, phase)) return true;
    return false;
}

// softcap * tanh(x / softcap) as softcap * (1 - 2 / (1 + exp(2x/softcap))).
// The hardware tanh's 2^-11 would move a capped score by 1e-2; this form's
// error is a few 2^-24 of the cap.  exp's overflow and underflow give the
// limits +-softcap.
__device__ __forceinline__ float cap_score(float x, float cap, float two_log2e_over_cap) {
    const float e = ex2f(x * two_log2e_over_cap);
    return fmaf(-2.0f * cap, rcpf(1.0f + e), cap);
}

// The score of one (query, key) pair in natural units; masks are the caller's.
// PRECISE: tanhf (float32 calls, whose other errors are as small as its own).
template <bool PRECISE>
__device__ __forceinline__ float attn_score(float dot, const ScoreArgs &s, float slope, int dist) {
    float x = dot * s.scale;
    if (s.cap > 0.0f) x = PRECISE ? s.cap * tanhf(x / s.cap) : cap_score(x, s.cap, s.cap_arg);
    if (s.bias) x = fmaf(-slope, (float)dist, x);
    return x;
}

// positions are >= 0: their difference fits
__device__ __forceinline__ int pos_dist(int qp, int kp) { return (int)((unsigned)qp - (unsigned)kp); }

// ---------------------------------------------------------------------------
// one request's keys
// ---------------------------------------------------------------------------
struct KeyRange {
    int lo, hi;   // keys [lo, hi): entries below `len`, then the candidates
    int len;      // committed entries
    bool ok;
};

// Request b's keys (mode 1: the shared prefix; mode 2: the committed entries,
// for the weights).  Entries that the window or the document's start hides
// from every query are left out where positions are indices.
__device__ __forceinline__ KeyRange attn_keys(const AttnParams &p, int b) {
    KeyRange r;
    if (p.mode == 1) {
        r.lo = 0;
        r.hi = r.len = p.P;
        r.ok = true;
        return r;
    }
    r.len = p.len[b];
    const int n = p.mode == 2 ? p.n_slots[b] : p.S;  // queries
    r.ok = r.len >= (p.mode == 2 ? 0 : p.P) &&
           (int64_t)r.len + (p.mode == 2 || p.tk ? 0 : p.S) <= (int64_t)p.max_blocks * p.bs;
    if (p.mode == 2) r.ok = r.ok && n >= 0 && n <= p.S && n <= r.len;
    if (!r.ok) {
        r.lo = r.hi = r.len = 0;
        return r;
    }
    r.hi = p.mode == 2 ? r.len : r.len + p.S;
    int64_t lo = p.P;
    if (!p.key_pos) {
        if (p.first) lo = max(lo, (int64_t)p.first[b]);
        if (p.window > 0) {
            int qmin = p.mode == 2 ? r.len - n : r.len;
            if (p.pos) {
                qmin = 0x7fffffff;
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int s = p.mode == 2 && p.slots ? p.slots[(int64_t)b * p.slots_stride + i] : i;
                    if (s >= 0 && s < p.S) qmin = min(qmin, p.pos[(int64_t)b * p.S + s]);
                }
            }
            lo = max(lo, (int64_t)qmin - p.window + 1);
        }
    }
    r.lo = (int)min(lo, (int64_t)(p.mode == 2 ? r.len - n : r.len));
    if (p.mode == 2) r.lo = n == 0 ? r.hi : min(max(r.lo, p.P), r.hi);
    return r;
}

// Where keys are copied in boxes of p.box rows of one page (p.box > 0), a tile
// line starts at a box boundary and the candidates begin a new box: `lo` is the
// first key of the line, `entries` the keys before the candidates.
struct KeyLine {
    int lo, entries;
};
__device__ __forceinline__ KeyLine attn_line(const AttnParams &p, const KeyRange &r) {
    KeyLine k;
    const int mask = ~(p.box - 1);  // (a power of two)
    k.lo = r.lo & mask;
    const int end = p.tk && p.mode == 0 ? r.len : r.hi;
    // (no entry in range: none is looked up, though `lo` may lie inside a page)
    k.entries = r.lo < end ? (end - k.lo + p.box - 1) & mask : 0;
    return k;
}

__device__ __forceinline__ int attn_tiles(const AttnParams &p, const KeyRange &r, int kt) {
    int n = r.hi - r.lo;
    if (p.box > 0 && r.ok) n = attn_line(p, r).entries + (p.tk && p.mode == 0 ? p.S : 0);
    return max(1, (n + kt - 1) / kt);
}

// ---------------------------------------------------------------------------
// the line of tiles
// ---------------------------------------------------------------------------
struct AttnPlan {
    int64_t total, share;       // tiles in all, tiles per block
    int64_t pre[kAttnThreadsMax + 1];  // tiles before the requests of thread t
    int chunk;                  // requests per thread
};

// Fills `pl` (shared memory); the first NT threads of the block call it.
// `per`: items of a request.
template <int NT> __device__ __forceinline__ void attn_plan(const AttnParams &p, AttnPlan &pl, int per, int kt) {
    const int tid = threadIdx.x;
    const int nreq = p.mode == 1 ? 1 : p.B;
    const int chunk = (nreq + NT - 1) / NT;
    int64_t sum = 0;
    for (int b = tid * chunk; b < min(nreq, (tid + 1) * chunk); ++b) sum += attn_tiles(p, attn_keys(p, b), kt);
    pl.pre[tid + 1] = sum * per;
    sync_nt<NT>();
    if (tid < 32) {  // inclusive scan by one warp, NT/32 values a lane
        constexpr int V = NT / 32;
        int64_t v[V], s = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s += pl.pre[tid * V + i + 1];
            v[i] = s;
        }
        int64_t inc = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(kFull, inc, o);
            if (tid >= o) inc += up;
        }
        const int64_t before = inc - s;
#pragma unroll
        for (int i = 0; i < V; ++i) pl.pre[tid * V + i + 1] = before + v[i];
        if (tid == 31) {
            pl.total = inc;
            const int64_t g = gridDim.x;
            pl.share = max((inc + g - 1) / g, (int64_t)p.min_share);
            pl.chunk = chunk;
            pl.pre[0] = 0;
        }
    }
    sync_nt<NT>();
}

struct AttnItem {
    int b, h, rt;          // request (0 in mode 1), cached head, row tile
    int64_t u0;            // its first tile on the line
    int ntiles;
    KeyRange keys;
};

// The item holding tile u (< total).  Uniform over the block.
template <int NT>
__device__ __forceinline__ AttnItem attn_find(const AttnParams &p, const AttnPlan &pl, int64_t u, int per, int rtiles, int kt) {
    int lo = 0, hi = NT;  // the last t with pre[t] <= u
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (pl.pre[m] <= u) lo = m; else hi = m;
    }
    AttnItem it;
    int64_t at = pl.pre[lo];
    const int nreq = p.mode == 1 ? 1 : p.B;
    int b = lo * pl.chunk;
    KeyRange r = attn_keys(p, b);
    int nt = attn_tiles(p, r, kt);
    while (at + (int64_t)nt * per <= u && b + 1 < nreq) {
        at += (int64_t)nt * per;
        r = attn_keys(p, ++b);
        nt = attn_tiles(p, r, kt);
    }
    const int k = (int)((u - at) / nt);
    it.b = b;
    it.h = k / rtiles;
    it.rt = k - it.h * rtiles;
    it.u0 = at + (int64_t)k * nt;
    it.ntiles = nt;
    it.keys = r;
    return it;
}

// the item after `it`
__device__ __forceinline__ AttnItem attn_next(const AttnParams &p, const AttnItem &it, int per, int rtiles, int kt) {
    AttnItem n = it;
    n.u0 += it.ntiles;
    if (++n.rt == rtiles) {
        n.rt = 0;
        if (++n.h == per / rtiles) {
            n.h = 0;
            ++n.b;
            n.keys = attn_keys(p, n.b);
            n.ntiles = attn_tiles(p, n.keys, kt);
        }
    }
    return n;
}

// ---------------------------------------------------------------------------
// one key's K (or V) row: where it lies, or null (past the end, a bad block)
// ---------------------------------------------------------------------------
// Element offset of entry c's row of cached head h in the layer's plane; -1
// for a block id out of range.
__device__ __forceinline__ int64_t entry_offset(const AttnParams &p, const int *table, int c, int h) {
    const int j = (int)fast_div((unsigned)c, p.bs_div);
    const int blk = __ldg(table + j);
    if (blk < 0 || (int64_t)blk >= p.nb) return -1;
    return (((int64_t)blk * p.bs + (c - j * p.bs)) * p.H + h) * p.D;
}

static __device__ __noinline__ void attn_flag(const AttnParams &p, int b) {
    atomicOr(p.status, SPEC_FLAG_BAD_INPUT);
    if (!p.flags) return;
    if (p.mode == 1) {
        for (int i = 0; i < p.B; ++i) atomicOr(p.flags + i, SPEC_FLAG_BAD_INPUT);
    } else {
        atomicOr(p.flags + b, SPEC_FLAG_BAD_INPUT);
    }
}

// One row tile's queries.
template <int RT> struct AttnRows {
    int qp[RT];        // position
    int first[RT];     // first position seen
    float slope[RT];
    int64_t out[RT];   // row of out / lse / the shared results; -1: no such row
    int64_t q[RT];     // element offset of the query
    int cand[RT];      // candidate index
};

// Row r of the item (mode 1: over all requests), by NT threads.
template <int RT, int NT>
__device__ __forceinline__ void attn_rows(const AttnParams &p, const AttnItem &it, AttnRows<RT> &w, int tid) {
    const int per = p.S * p.G;
    const int64_t nrows = p.mode == 1 ? (int64_t)p.B * per : per;
    for (int i = tid; i < RT; i += NT) {
        const int64_t r = (int64_t)it.rt * RT + i;
        if (r >= nrows) {
            w.out[i] = w.q[i] = -1;
            w.qp[i] = w.cand[i] = 0;
            w.first[i] = 0;
            w.slope[i] = 0.0f;
            continue;
        }
        const int b = p.mode == 1 ? (int)(r / per) : it.b;
        const int k = p.mode == 1 ? (int)(r - (int64_t)b * per) : (int)r;
        const int s = k / p.G, hq = it.h * p.G + (k - s * p.G);
        w.cand[i] = s;
        w.qp[i] = p.pos ? p.pos[(int64_t)b * p.S + s] : p.len[b] + s;
        w.first[i] = p.first ? p.first[b] : (int)0x80000000;
        w.slope[i] = p.slopes ? p.slopes[hq] : 0.0f;
        w.out[i] = ((int64_t)b * p.S + s) * p.Hq + hq;
        w.q[i] = b * p.qsb + s * p.qss + hq * p.qsh;
    }
}

// Whether key c (index; position kp) may be seen by row i.
template <int RT>
__device__ __forceinline__ bool attn_visible(const AttnParams &p, const AttnItem &it, const AttnRows<RT> &w, int i,
                                             int c, int kp, int dist) {
    bool v = kp >= w.first[i] && (p.window == 0 || dist < p.window);
    if (p.mode == 0 && c >= it.keys.len) {
        const int j = c - it.keys.len, s = w.cand[i];
        v = v && (p.mask ? (p.mask[((int64_t)it.b * p.S + s) * p.W + (j >> 5)] >> (j & 31)) & 1u : j <= s);
    }
    return v;
}

__device__ __forceinline__ int key_position(const AttnParams &p, const AttnItem &it, int c) {
    if (p.mode == 1) return c;
    if (c >= it.keys.len) {
        const int j = c - it.keys.len;
        return p.pos ? p.pos[(int64_t)it.b * p.S + j] : c;
    }
    return p.key_pos ? p.key_pos[(int64_t)it.b * p.kps + c] : c;
}

// Mode 2, a request's first tile, its slots good: the positions of the committed
// candidates whose entries lie among the shared ones, which no tile holds (threads
// `tid` of `nt`).
__device__ __forceinline__ void shared_positions(const WeightsParams &wp, const AttnItem &it, int tid, int nt) {
    const AttnParams &p = wp.a;
    if (!wp.key_pos_out) return;
    const int cand0 = it.keys.len - p.n_slots[it.b];
    for (int c = cand0 + tid; c < it.keys.lo; c += nt) {
        const int j = c - cand0, s = p.slots ? p.slots[(int64_t)it.b * p.slots_stride + j] : j;
        wp.key_pos_out[(int64_t)it.b * p.kps + c] = p.pos ? p.pos[(int64_t)it.b * p.S + s] : c;
    }
}

// ---------------------------------------------------------------------------
// results
// ---------------------------------------------------------------------------
template <typename T> __device__ __forceinline__ void store4(T *p, float4 v);
template <> __device__ __forceinline__ void store4<float>(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 u = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
    *reinterpret_cast<uint2 *>(p) = u;
}

// 2^(a - m) for a <= m; 0 for a = -inf, m = -inf included
__device__ __forceinline__ float rel_weight(float a, float m) { return a == -INFINITY ? 0.0f : ex2f(a - m); }

// What attn_write needs of the shared part, loaded ahead.
struct SharedPart {
    float lse;
    float4 o;
};
__device__ __forceinline__ SharedPart attn_shared_part(const AttnParams &p, bool ok, int64_t row, int d) {
    SharedPart s{-INFINITY, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (p.mode == 0 && p.P > 0 && ok && row >= 0) {
        s.lse = p.pre_lse[row];
        s.o = *reinterpret_cast<const float4 *>(p.pre_o + row * p.D + d);
    }
    return s;
}

// Writes four columns of row `row` from the joined (m2, l, o): to the shared
// results in mode 1, else to the output, the shared part joined first (not for
// a request whose length is bad: it gets zeros).
template <typename T>
__device__ __forceinline__ void attn_write(const AttnParams &p, bool ok, int64_t row, int d, float m2, float l,
                                           float4 o, const SharedPart &sp) {
    float lse2 = l > 0.0f || l != l ? m2 + lg2f(l) : -INFINITY;  // a NaN sum stays NaN
    if (p.mode == 1) {
        const float inv = lse2 == -INFINITY ? 0.0f : 1.0f / l;
        *reinterpret_cast<float4 *>(p.pre_o + row * p.D + d) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (d == 0) p.pre_lse[row] = lse2;
        return;
    }
    if (p.P > 0 && ok) {
        const float m = fmaxf(m2, sp.lse);
        const float a = rel_weight(m2, m), c = sp.lse != sp.lse ? sp.lse : rel_weight(sp.lse, m);
        l = l * a + c;
        o = make_float4(o.x * a + sp.o.x * c, o.y * a + sp.o.y * c, o.z * a + sp.o.z * c, o.w * a + sp.o.w * c);
        lse2 = l > 0.0f || l != l ? m + lg2f(l) : -INFINITY;
    }
    const float inv = lse2 == -INFINITY ? 0.0f : 1.0f / l;
    if (lse2 == -INFINITY) o = make_float4(0.f, 0.f, 0.f, 0.f);
    store4(static_cast<T *>(p.out) + row * p.D + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (d == 0 && p.lse) p.lse[row] = lse2 * kLn2;
}

// Whether the item lies in several blocks, and which.
struct ItemBlocks {
    int c0, c1;
};
__device__ __forceinline__ ItemBlocks attn_blocks(const AttnPlan &pl, const AttnItem &it) {
    // mostly this block alone: no division then
    const int64_t mine = (int64_t)blockIdx.x * pl.share;
    if (it.u0 >= mine && it.u0 + it.ntiles <= mine + pl.share) return ItemBlocks{(int)blockIdx.x, (int)blockIdx.x};
    return ItemBlocks{(int)(it.u0 / pl.share), (int)((it.u0 + it.ntiles - 1) / pl.share)};
}
// Block c's partial result: slot 0 of a block holds the item that began before
// it, slot 1 the one that goes on after it.  RT rows of D sums, references,
// weights.
template <int RT> __device__ __forceinline__ float *attn_part(const AttnParams &p, int c, int c0) {
    return p.part + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * ((int64_t)RT * (p.D + 2));
}

// Query r (of the item's RT rows) joined by a warp from the partial results of n
// blocks, from block c0 on:
//   m = max m_c, l = sum l_c 2^(m_c - m), o = sum o_c 2^(m_c - m)
// A lane takes four columns; U blocks' rows are in flight.  NANS: sums that are NaN show
// from a block whose weight is 0 too.
template <typename T, int U, bool NANS = false>
__device__ __forceinline__ void attn_join_row(const AttnParams &p, bool ok, int rt_rows, int c0, int n, int r, int64_t row) {
    const int lane = threadIdx.x & 31;
    const int64_t slot = (int64_t)rt_rows * (p.D + 2), o_m = (int64_t)rt_rows * p.D, o_l = o_m + rt_rows;
    const float *base = p.part + (int64_t)c0 * 2 * slot;
    auto part = [&](int c) { return base + (int64_t)c * 2 * slot + (c == 0 ? slot : 0); };
    // the first blocks' rows, references and weights in one round
    float mc = -INFINITY, lc = 0.0f;
    if (lane < n) {
        mc = __ldcg(part(lane) + o_m + r);
        lc = __ldcg(part(lane) + o_l + r);
    }
#pragma unroll 1
    for (int d0 = 0; d0 < p.D; d0 += 128) {
        const int d = d0 + lane * 4;
        const bool in = d < p.D;
        const SharedPart sp = attn_shared_part(p, ok && in, row, in ? d : 0);
        float4 x[U];
        auto load = [&](int c0) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                x[i] = c0 + i < n && in ? __ldcg(reinterpret_cast<const float4 *>(part(c0 + i) + (int64_t)r * p.D + d))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        load(0);
        float m = mc;
        for (int c = lane + 32; c < n; c += 32) m = fmaxf(m, __ldcg(part(c) + o_m + r));
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, k));
        float l = 0.0f, w = 0.0f, lw = 0.0f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < n; c += U) {
            if ((c & 31) == 0) {  // the weights of the next 32 blocks (0: no key of the row, NaN scores alone, or far below)
                const bool mine = c + lane < n;
                const float a = c == 0 ? mc : mine ? __ldcg(part(c + lane) + o_m + r) : -INFINITY;
                const float b = c == 0 ? lc : mine ? __ldcg(part(c + lane) + o_l + r) : 0.0f;
                w = mine ? rel_weight(a, m) : 0.0f;
                lw = b * w;  // (a NaN sum stays one: its block saw a NaN score)
            }
            if (c > 0) load(c);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float wc = __shfl_sync(kFull, w, (c + i) & 31);
                l += __shfl_sync(kFull, lw, (c + i) & 31);
                if (NANS || wc != 0.0f)
                    o = make_float4(fmaf(x[i].x, wc, o.x), fmaf(x[i].y, wc, o.y), fmaf(x[i].z, wc, o.z), fmaf(x[i].w, wc, o.w));
            }
        }
        if (in) attn_write<T>(p, ok, row, d, m, l, o, sp);
    }
}

// After this block's partial result has been stored (NT threads): the block
// that arrives last joins the item.  The counter is left zero.
template <typename T, int RT, int NT, bool NANS>
__device__ __forceinline__ void attn_join_here(const AttnParams &p, const AttnItem &it, const AttnRows<RT> &w, ItemBlocks ib,
                                               int *last) {
    const int tid = threadIdx.x, n = ib.c1 - ib.c0 + 1;
    __threadfence();
    sync_nt<NT>();
    if (tid == 0) *last = atomicAdd(p.counters + ib.c0, 1u) == (unsigned)(n - 1);
    sync_nt<NT>();
    if (!*last) return;
    __threadfence();
    for (int r = tid >> 5; r < RT; r += NT / 32)
        if (w.out[r] >= 0) attn_join_row<T, 8, NANS>(p, it.keys.ok, RT, ib.c0, n, r, w.out[r]);
    if (tid == 0) p.counters[ib.c0] = 0u;
    sync_nt<NT>();
}

// For the second kernel: marks the item that begins in this block and goes on in
// others (thread 0; attn_begin has marked the block as having none).
__device__ __forceinline__ void attn_begin(const AttnParams &p) {
    if (threadIdx.x == 0) p.split[blockIdx.x].blocks = 0;
}
__device__ __forceinline__ void attn_mark(const AttnParams &p, const AttnItem &it, ItemBlocks ib) {
    if (threadIdx.x == 0 && (int)blockIdx.x == ib.c0)
        p.split[ib.c0] = SplitItem{ib.c1 - ib.c0 + 1, it.b, it.h, it.rt, it.keys.ok ? 1 : 0};
}

// The block's result for item `it`, in shared memory: sums so[RT][ld] with
// reference m2 = sm[r] (log2 units) and weight sl[r].  Ends with the shared
// memory free for reuse.  A split item is joined by the block that arrives last.
template <typename T, int RT, int NT, bool NANS = false>
__device__ __forceinline__ void attn_finish(const AttnParams &p, const AttnPlan &pl, const AttnItem &it,
                                            const AttnRows<RT> &w, const float *so, int ld, const float *sm,
                                            const float *sl, int *last) {
    const int tid = threadIdx.x, lane = tid & 31;
    const ItemBlocks ib = attn_blocks(pl, it);
    const bool split = ib.c0 != ib.c1;
    float *mine = attn_part<RT>(p, blockIdx.x, ib.c0);
    // a warp per row, the shared part of four rows in flight
    constexpr int NW = NT / 32, U = 4;
#pragma unroll 1
    for (int r0 = tid >> 5; r0 < RT; r0 += NW * U)
#pragma unroll 1
        for (int d = lane * 4; d < p.D; d += 128) {
            SharedPart sp[U];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const int r = r0 + q * NW;
                sp[q] = attn_shared_part(p, it.keys.ok && !split, r < RT ? w.out[r] : -1, d);
            }
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const int r = r0 + q * NW;
                if (r >= RT || w.out[r] < 0) continue;
                const float4 v = *reinterpret_cast<const float4 *>(so + r * ld + d);
                if (split) __stcg(reinterpret_cast<float4 *>(mine + (int64_t)r * p.D + d), v);
                else attn_write<T>(p, it.keys.ok, w.out[r], d, sm[r], sl[r], v, sp[q]);
            }
        }
    if (split) {
        for (int r = tid; r < RT; r += NT) {
            __stcg(mine + (int64_t)RT * p.D + r, sm[r]);
            __stcg(mine + (int64_t)RT * p.D + RT + r, sl[r]);
        }
        attn_join_here<T, RT, NT, NANS>(p, it, w, ib, last);
    } else {
        sync_nt<NT>();
    }
}

// The same for a kernel whose thread holds a whole row: (m2, l) and, by
// `chunk(d, o)`, 32 columns from d on (every lane of a warp calls it together).
// `r`: the thread's row in the item's tile of RT rows.  A split item is left to the
// second kernel.
template <typename T, int RT, int NT, typename F>
__device__ __forceinline__ void attn_finish_row(const AttnParams &p, const AttnPlan &pl, const AttnItem &it,
                                                const AttnRows<RT> &w, int r, float m, float l, F &&chunk) {
    const ItemBlocks ib = attn_blocks(pl, it);
    const bool split = ib.c0 != ib.c1;
    const int64_t out_row = w.out[r];
    float *mine = attn_part<RT>(p, blockIdx.x, ib.c0);
#pragma unroll 1
    for (int d0 = 0; d0 < p.D; d0 += 32) {
        float o[32];
        chunk(d0, o);
        if (out_row < 0) continue;
        SharedPart sp[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = d0 + 4 * j;
            if (d >= p.D) break;
            if (j % 4 == 0 && !split) {
#pragma unroll
                for (int q = 0; q < 4; ++q) sp[q] = attn_shared_part(p, it.keys.ok && d + 4 * q < p.D, out_row, d + 4 * q);
            }
            const float4 v = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            if (split) __stcg(reinterpret_cast<float4 *>(mine + (int64_t)r * p.D + d), v);
            else attn_write<T>(p, it.keys.ok, out_row, d, m, l, v, sp[j % 4]);
        }
    }
    if (!split) return;
    __stcg(mine + (int64_t)RT * p.D + r, m);
    __stcg(mine + (int64_t)RT * p.D + RT + r, l);
    attn_mark(p, it, ib);
}

}  // namespace specv
