// Shared device code of the paged-cache attention kernels (sm_103a): the
// score, the split of the work over the grid, and the join of split results.
//
// Work.  A tile is `kt` consecutive keys; an item is a (request, cached head,
// row tile) with its keys in tiles, rows being the S * Hq/H queries that share
// the cached head.  The pass over a shared prefix is one request whose rows
// are every request's.  All items' tiles form one line; block i takes tiles
// [i*share, (i+1)*share), so lengths from one token to the longest give every
// block the same work.  An item that lies in several blocks is joined by the
// block that arrives last, from all blocks' partial results in block order:
// the result does not depend on which block that is.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace specv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// softcap * tanh(x / softcap) as softcap * (1 - 2 / (1 + exp(2x/softcap))).
// The hardware tanh's 2^-11 would move a capped score by 1e-2; this form's
// error is a few 2^-24 of the cap.  exp's overflow and underflow give the
// limits +-softcap.
__device__ __forceinline__ float cap_score(float x, float cap, float two_log2e_over_cap) {
    const float e = ex2f(x * two_log2e_over_cap);
    return fmaf(-2.0f * cap, __fdividef(1.0f, 1.0f + e), cap);
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
    const int box = p.box;
    k.lo = r.lo / box * box;
    const int end = p.tk && p.mode == 0 ? r.len : r.hi;
    k.entries = (end - k.lo + box - 1) / box * box;
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

// Writes four columns of row `row` from the joined (m2, l, o): to the shared
// results in mode 1, else to the output, the shared part joined first (not for
// a request whose length is bad: it gets zeros).
template <typename T>
__device__ __forceinline__ void attn_write(const AttnParams &p, bool ok, int64_t row, int d, float m2, float l,
                                           float4 o) {
    float lse2 = l > 0.0f || l != l ? m2 + lg2f(l) : -INFINITY;  // a NaN sum stays NaN
    if (p.mode == 1) {
        const float inv = lse2 == -INFINITY ? 0.0f : 1.0f / l;
        *reinterpret_cast<float4 *>(p.pre_o + row * p.D + d) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (d == 0) p.pre_lse[row] = lse2;
        return;
    }
    if (p.P > 0 && ok) {
        const float ls = p.pre_lse[row];
        const float4 os = *reinterpret_cast<const float4 *>(p.pre_o + row * p.D + d);
        const float m = fmaxf(m2, ls);
        const float a = rel_weight(m2, m), c = ls != ls ? ls : rel_weight(ls, m);
        l = l * a + c;
        o = make_float4(o.x * a + os.x * c, o.y * a + os.y * c, o.z * a + os.z * c, o.w * a + os.w * c);
        lse2 = l > 0.0f || l != l ? m + lg2f(l) : -INFINITY;
    }
    const float inv = lse2 == -INFINITY ? 0.0f : 1.0f / l;
    if (lse2 == -INFINITY) o = make_float4(0.f, 0.f, 0.f, 0.f);
    store4(static_cast<T *>(p.out) + row * p.D + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (d == 0 && p.lse) p.lse[row] = lse2 * kLn2;
}

// The block's result for item `it`, in shared memory: sums so[RT][ld] with
// reference m2 = sm[r] (log2 units) and weight sl[r].  [t0, t1) are the tiles
// this block did.  Ends with the shared memory free for reuse.
template <typename T, int RT, int NT>
__device__ __forceinline__ void attn_finish(const AttnParams &p, const AttnPlan &pl, const AttnItem &it,
                                            const AttnRows<RT> &w, const float *so, int ld, const float *sm,
                                            const float *sl, int *last_flag) {
    const int tid = threadIdx.x, d4 = p.D / 4;
    const int64_t share = pl.share;
    const int c0 = (int)(it.u0 / share), c1 = (int)((it.u0 + it.ntiles - 1) / share);
    if (c0 == c1) {
        for (int i = tid; i < RT * d4; i += NT) {
            const int r = i / d4, d = (i - r * d4) * 4;
            if (w.out[r] >= 0)
                attn_write<T>(p, it.keys.ok, w.out[r], d, sm[r], sl[r], *reinterpret_cast<const float4 *>(so + r * ld + d));
        }
        sync_nt<NT>();
        return;
    }
    // partial results: slot 0 of a block holds the item that began before it,
    // slot 1 the one that goes on after it
    const int64_t slot_floats = (int64_t)RT * (p.D + 2);
    const int me = blockIdx.x;
    float *mine = p.part + ((int64_t)me * 2 + (me == c0 ? 1 : 0)) * slot_floats;
    for (int i = tid; i < RT * d4; i += NT) {
        const int r = i / d4, d = (i - r * d4) * 4;
        if (w.out[r] >= 0) __stcg(reinterpret_cast<float4 *>(mine + r * p.D + d), *reinterpret_cast<const float4 *>(so + r * ld + d));
    }
    for (int r = tid; r < RT; r += NT) {
        __stcg(mine + RT * p.D + r, sm[r]);
        __stcg(mine + RT * p.D + RT + r, sl[r]);
    }
    __threadfence();
    sync_nt<NT>();
    if (tid == 0) *last_flag = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
    sync_nt<NT>();
    if (!*last_flag) return;
    __threadfence();
    // a warp per row: each lane a few blocks' (m, l), then the rows, many in flight
    const int lane = tid & 31, n = c1 - c0 + 1;
    auto part = [&](int c) { return p.part + ((int64_t)(c0 + c) * 2 + (c == 0 ? 1 : 0)) * slot_floats; };
    for (int r = tid >> 5; r < RT; r += NT / 32) {
        if (w.out[r] < 0) continue;
        constexpr int U = 8;
        float m = -INFINITY;
        for (int c = lane; c < n; c += 32) m = fmaxf(m, __ldcg(part(c) + RT * p.D + r));
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, x));
        for (int d = lane * 4; d < p.D + (128 - p.D % 128) % 128; d += 128) {  // all lanes stay
            float l = 0.0f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int cb = 0; cb < n; cb += 32) {
                float k = 0.0f, lk = 0.0f;
                if (cb + lane < n) {
                    k = rel_weight(__ldcg(part(cb + lane) + RT * p.D + r), m);
                    lk = __ldcg(part(cb + lane) + RT * p.D + RT + r) * k;
                    if (k == 0.0f) lk = 0.0f;  // that block saw no key of the row
                }
                const int e = min(32, n - cb);
                for (int c = 0; c < e; c += U) {
                    float4 x[U];
#pragma unroll
                    for (int q = 0; q < U; ++q)
                        x[q] = c + q < e && d < p.D ? __ldcg(reinterpret_cast<const float4 *>(part(cb + c + q) + (int64_t)r * p.D + d))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int q = 0; q < U; ++q) {
                        const float kq = __shfl_sync(kFull, k, (c + q) & 31);
                        l += __shfl_sync(kFull, c + q < e ? lk : 0.0f, (c + q) & 31);
                        if (c + q < e && kq != 0.0f)
                            o = make_float4(fmaf(x[q].x, kq, o.x), fmaf(x[q].y, kq, o.y), fmaf(x[q].z, kq, o.z), fmaf(x[q].w, kq, o.w));
                    }
                }
            }
            if (d < p.D) attn_write<T>(p, it.keys.ok, w.out[r], d, m, l, o);
        }
    }
    if (tid == 0) p.counters[c0] = 0u;
    sync_nt<NT>();
}

// The same for a kernel whose thread holds a whole row: (m2, l) and, by
// `chunk(d, o)`, 32 columns from d on (every lane of a warp calls it together).
// `r`: the thread's row in the item's tile of RT rows.
template <typename T, int RT, int NT, typename F>
__device__ __forceinline__ void attn_finish_row(const AttnParams &p, const AttnPlan &pl, const AttnItem &it,
                                                int64_t out_row, int r, float m, float l, F &&chunk, int *last_flag) {
    const int64_t share = pl.share;
    const int c0 = (int)(it.u0 / share), c1 = (int)((it.u0 + it.ntiles - 1) / share);
    const bool split = c0 != c1;
    const int64_t slot_floats = (int64_t)RT * (p.D + 2);
    const int me = blockIdx.x;
    float *mine = p.part + ((int64_t)me * 2 + (me == c0 ? 1 : 0)) * slot_floats;
    for (int d0 = 0; d0 < p.D; d0 += 32) {
        float o[32];
        chunk(d0, o);
        if (out_row < 0) continue;
#pragma unroll
        for (int d = 0; d < 32; d += 4) {
            if (d0 + d >= p.D) break;
            const float4 v = make_float4(o[d], o[d + 1], o[d + 2], o[d + 3]);
            if (split) __stcg(reinterpret_cast<float4 *>(mine + (int64_t)r * p.D + d0 + d), v);
            else attn_write<T>(p, it.keys.ok, out_row, d0 + d, m, l, v);
        }
    }
    if (!split) return;
    __stcg(mine + RT * p.D + r, m);
    __stcg(mine + RT * p.D + RT + r, l);
    __threadfence();
    sync_nt<NT>();
    if (threadIdx.x == 0) *last_flag = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
    sync_nt<NT>();
    if (!*last_flag) return;
    __threadfence();
    if (out_row >= 0) {
        float mm = -INFINITY;
        for (int c = c0; c <= c1; ++c)
            mm = fmaxf(mm, __ldcg(p.part + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * slot_floats + RT * p.D + r));
        for (int d0 = 0; d0 < p.D; d0 += 32) {
            float4 o[8];
            float ll = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = c0; c <= c1; ++c) {
                const float *s = p.part + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * slot_floats;
                const float k = rel_weight(__ldcg(s + RT * p.D + r), mm);
                if (k == 0.0f) continue;  // this block saw no key of the row
                ll += __ldcg(s + RT * p.D + RT + r) * k;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (d0 + 4 * j >= p.D) break;
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(s + (int64_t)r * p.D + d0 + 4 * j));
                    o[j] = make_float4(fmaf(x.x, k, o[j].x), fmaf(x.y, k, o[j].y), fmaf(x.z, k, o[j].z), fmaf(x.w, k, o[j].w));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (d0 + 4 * j < p.D) attn_write<T>(p, it.keys.ok, out_row, d0 + 4 * j, mm, ll, o[j]);
        }
    }
    if (threadIdx.x == 0) p.counters[c0] = 0u;
    sync_nt<NT>();
}

}  // namespace specv
