// The 8-bit cache's writer, reader and the commit of a tree's path
// (spec_write_kv_q8, spec_read_kv_q8, spec_commit_kv_q8); its numbers: kv8.cuh.
//
// Writing and reading: a block has 16 or 64 entries and up to 32 heads of K or V, a
// group of lanes a row, 16 values a lane where they are written and 8 where they are
// read; a row's largest magnitude is a few shuffles.  The rows' exponents lie a head's
// next to each other, so that attention reads a page's in one piece: they pass
// through shared memory and leave a head's entries together.  64 entries where that
// gives every SM two blocks (fewer look-ups and starts: prompts read back 117 us
// instead of 145), else 16.
// Measured: 65,600 entries of 8 heads of 128, bf16 parts of a fused projection's
// output, written in 81 us (4.9 TB/s; with 8 values a lane 98, bound by issue), as
// many read back, 8,192 a request with zeros, in 117 us (5.8 TB/s).  Both are bound by
// HBM and by what a row costs besides.
//
// Commit: a kept candidate's codes and exponents move from entry len + slots[i] to
// len + i.  slots ascend, so slots[i] >= i, and a place is read before, or in the
// same batch of loads as, it is written: a thread that takes the same 16 bytes of
// all entries in order needs to wait for nobody.
#include "attn_params.h"
#include "common.cuh"
#include "kv8.cuh"

#include <type_traits>

namespace specv {
namespace {

constexpr int kHeads = 32, kThreads = 256;

struct Place {
    int64_t entry;  // blk * bs + offset, or -1
    int64_t scale;  // of head 0's exponent; another head's lies bs further on
};

// The place of entry c of request b; flags a block id out of range.
__device__ __forceinline__ Place place_of(const Kv8Params &p, int b, int c) {
    const int j = (int)fast_div((unsigned)c, p.bs_div), off = c - j * p.bs;
    const int blk = __ldg(p.table + (int64_t)b * p.max_blocks + j);
    if (blk < 0 || (int64_t)blk >= p.nb) {
        if (p.flags) atomicOr(p.flags + b, SPEC_FLAG_BAD_INPUT);
        atomicOr(p.status, SPEC_FLAG_BAD_INPUT);
        return Place{-1, 0};
    }
    return Place{(int64_t)blk * p.bs + off, (int64_t)blk * p.H * p.bs + off};
}

// the larger, or NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 values of a row; their largest magnitude (NaN if one is); their codes
template <typename T> struct Raw16;
template <> struct Raw16<__nv_bfloat16> {
    uint4 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        v[0] = ld_nc16(p);
        v[1] = ld_nc16(p + 8);
    }
    __device__ __forceinline__ float top() const {
        uint32_t a = 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            constexpr uint32_t m = 0x7fff7fffu;
            a = max_nan2(a, max_nan2(max_nan2(v[i].x & m, v[i].y & m), max_nan2(v[i].z & m, v[i].w & m)));
        }
        return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    }
    __device__ __forceinline__ void values(int i, float *x) const { unpack<__nv_bfloat16>(v[i], x); }
};
template <> struct Raw16<float> {
    uint4 v[4];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ld_nc16(p + 4 * i);
    }
    __device__ __forceinline__ float top() const {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4];
            unpack<float>(v[i], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) a = max_nan(a, fabsf(x[e]));
        }
        return a;
    }
    __device__ __forceinline__ void values(int i, float *x) const {  // 8 of them
        unpack<float>(v[2 * i], x);
        unpack<float>(v[2 * i + 1], x + 4);
    }
};
__device__ __forceinline__ void store8(float *to, const float *x) {
    *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *to, const float *x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
    *reinterpret_cast<uint4 *>(to) = make_uint4(u[0], u[1], u[2], u[3]);
}

struct Tile {
    int b, e0, h0, heads, kv;
};
// Blocks: K/V fastest, then head chunks, E entries, requests.
template <int E> __device__ __forceinline__ Tile tile_of(const Kv8Params &p) {
    Tile t;
    int64_t i = blockIdx.x;
    t.kv = (int)(i & 1);
    i >>= 1;
    const int chunks = (p.H + kHeads - 1) / kHeads;
    t.h0 = (int)(i % chunks) * kHeads;
    i /= chunks;
    t.heads = min(kHeads, p.H - t.h0);
    t.e0 = (int)(i % p.etiles) * E;
    t.b = (int)(i / p.etiles);
    return t;
}

// G: lanes of a row
template <typename T, int G, int E> __global__ void __launch_bounds__(kThreads) write_kv8_kernel(Kv8Params p) {
    __shared__ Place place[E];
    __shared__ unsigned char scale[kHeads][E];
    const Tile t = tile_of<E>(p);
    const int tid = threadIdx.x;
    const int len = p.start[t.b], n = p.count ? p.count[t.b] : p.S;
    const bool good = len >= 0 && n >= 0 && n <= p.S && (int64_t)len + n <= (int64_t)p.max_blocks * p.bs;
    if (!good) {
        if (t.e0 == 0 && t.h0 == 0 && t.kv == 0 && tid == 0) {
            if (p.flags) atomicOr(p.flags + t.b, SPEC_FLAG_BAD_INPUT);
            atomicOr(p.status, SPEC_FLAG_BAD_INPUT);
        }
        return;
    }
    const int entries = min(E, n - t.e0);
    if (entries <= 0) return;
    constexpr int NG = kThreads / G;
    const int d = (tid % G) * 16, rows = entries * t.heads;
    const bool in = d < p.D;
    // row r of the block: entry, head
    auto at = [&](int r, int &e, int &h) {
        e = r / t.heads;
        h = r - e * t.heads;
        return r < rows;
    };
    const T *src = static_cast<const T *>(t.kv ? p.v : p.k) + t.b * p.sb[t.kv];
    unsigned char *codes = p.codes + (t.kv ? p.plane : 0);
    Raw16<T> raw;
    auto load = [&](int r) {
        int e, h;
        if (at(r, e, h) && in) raw.load(src + (t.e0 + e) * p.ss[t.kv] + (t.h0 + h) * p.sh[t.kv] + d);
    };
    load(tid / G);  // (the first rows are on their way while the blocks are looked up)
    if (tid < entries) place[tid] = place_of(p, t.b, len + t.e0 + tid);
    __syncthreads();
    for (int base = 0; base < rows; base += NG) {  // (every lane takes part in the shuffles)
        const int r = base + tid / G;
        if (base > 0) load(r);
        int e, h;
        const bool is = at(r, e, h);
        float top = is && in ? raw.top() : 0.0f;
#pragma unroll
        for (int q = G / 2; q > 0; q >>= 1) top = max_nan(top, __shfl_xor_sync(kFull, top, q));
        if (!is) continue;
        const unsigned s = kv8_scale(top);
        if (d == 0) scale[h][e] = (unsigned char)s;
        if (!in || place[e].entry < 0) continue;
        uint32_t c[4] = {0u, 0u, 0u, 0u};
        if (s != 255u) {
            const float f = kv8_inverse(s);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x[8];
                raw.values(i, x);
                c[2 * i] = kv8_code2(x[0] * f, x[1] * f) | kv8_code2(x[2] * f, x[3] * f) << 16;
                c[2 * i + 1] = kv8_code2(x[4] * f, x[5] * f) | kv8_code2(x[6] * f, x[7] * f) << 16;
            }
        }
        *reinterpret_cast<uint4 *>(codes + (place[e].entry * p.H + t.h0 + h) * p.D + d) = make_uint4(c[0], c[1], c[2], c[3]);
    }
    __syncthreads();
    unsigned char *sc = p.scale + (t.kv ? p.splane : 0);
    for (int i = tid; i < t.heads * E; i += kThreads) {
        const int h = i / E, e = i - h * E;
        if (e < entries && place[e].entry >= 0) sc[place[e].scale + (int64_t)(t.h0 + h) * p.bs] = scale[h][e];
    }
}

template <typename T, int G, int E> __global__ void __launch_bounds__(kThreads) read_kv8_kernel(Kv8Params p) {
    __shared__ Place place[E];
    __shared__ float power[kHeads][E];
    const Tile t = tile_of<E>(p);
    const int tid = threadIdx.x;
    const int start = p.start ? p.start[t.b] : 0, n = p.count ? p.count[t.b] : p.S;
    const bool good = start >= 0 && n >= 0 && n <= p.S && (int64_t)start + n <= (int64_t)p.max_blocks * p.bs;
    if (!good && t.e0 == 0 && t.h0 == 0 && t.kv == 0 && tid == 0) {
        if (p.flags) atomicOr(p.flags + t.b, SPEC_FLAG_BAD_INPUT);
        atomicOr(p.status, SPEC_FLAG_BAD_INPUT);
    }
    const int entries = min(E, p.S - t.e0), held = good ? min(entries, n - t.e0) : 0;
    if (tid < entries) place[tid] = tid < held ? place_of(p, t.b, start + t.e0 + tid) : Place{-1, 0};
    __syncthreads();
    const unsigned char *sc = p.scale + (t.kv ? p.splane : 0), *codes = p.codes + (t.kv ? p.plane : 0);
    for (int i = tid; i < t.heads * E; i += kThreads) {
        const int h = i / E, e = i - h * E;
        if (e < entries && place[e].entry >= 0)
            power[h][e] = kv8_power(__ldg(sc + place[e].scale + (int64_t)(t.h0 + h) * p.bs));
    }
    __syncthreads();
    constexpr int NG = kThreads / G, U = 8;
    const int d = (tid % G) * 8, rows = entries * t.heads;
    if (d >= p.D) return;
    auto at = [&](int r, int &e, int &h) {
        e = r / t.heads;
        h = r - e * t.heads;
        return r < rows;
    };
    T *out = static_cast<T *>(t.kv ? p.out_v : p.out_k) + ((int64_t)t.b * p.S + t.e0) * p.H * p.D;
    for (int r0 = tid / G; r0 < rows; r0 += NG * U) {
        uint2 c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int e, h;
            c[u] = make_uint2(0u, 0u);
            if (at(r0 + u * NG, e, h) && place[e].entry >= 0)
                c[u] = __ldg(reinterpret_cast<const uint2 *>(codes + (place[e].entry * p.H + t.h0 + h) * p.D + d));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int e, h;
            if (!at(r0 + u * NG, e, h)) continue;
            const float f = place[e].entry >= 0 ? power[h][e] : 0.0f;
            const float4 a = kv8_value4(c[u].x), b = kv8_value4(c[u].y);
            const float x[8] = {a.x * f, a.y * f, a.z * f, a.w * f, b.x * f, b.y * f, b.z * f, b.w * f};
            store8(out + ((int64_t)e * p.H + t.h0 + h) * p.D + d, x);
        }
    }
}

int64_t row_blocks(int32_t B, int32_t S, int32_t H, int E) {
    return (int64_t)B * ((S + E - 1) / E) * ((H + kHeads - 1) / kHeads) * 2;
}

constexpr int kCommitThreads = 128, kCommitUnits = kCommitThreads / 32;

__global__ void __launch_bounds__(kCommitThreads) commit_kv8_kernel(Kv8Params p) {
    extern __shared__ int64_t moves[];  // source and destination of slot i: entry, exponent
    const int b = blockIdx.x / p.etiles, grp = blockIdx.x - b * p.etiles;
    const int tid = threadIdx.x, lane = tid & 31;
    const int len = p.len[b], n = p.count[b];
    bool good = n >= 0 && n <= p.S && len >= 0 && (int64_t)len + n <= (int64_t)p.max_blocks * p.bs;
    Place *src = reinterpret_cast<Place *>(moves), *dst = src + p.S;
    if (good && p.slots) {
        const int *slots = p.slots + (int64_t)b * p.slots_stride;
        for (int i = tid; i < n; i += kCommitThreads) {
            const int s = slots[i];
            bool ok = s >= i && s < p.S && (i == 0 || slots[i - 1] < s) && (int64_t)len + s < (int64_t)p.max_blocks * p.bs;
            src[i].entry = -1;  // already in its place
            if (ok && s != i) {
                src[i] = place_of(p, b, len + s);
                dst[i] = place_of(p, b, len + i);
                ok = src[i].entry >= 0 && dst[i].entry >= 0;
            }
            good = good && ok;
        }
    }
    good = __syncthreads_and(good);
    if (!good) {
        if (grp == 0 && tid == 0) {
            if (p.flags) atomicOr(p.flags + b, SPEC_FLAG_BAD_INPUT);
            atomicOr(p.status, SPEC_FLAG_BAD_INPUT);
        }
        return;
    }
    const int unit = grp * kCommitUnits + (tid >> 5);
    if (p.slots && unit < (int64_t)2 * p.L) {
        unsigned char *codes = p.codes + (int64_t)unit * p.plane, *sc = p.scale + (int64_t)unit * p.splane;
        const int64_t bytes = (int64_t)p.H * p.D;
        constexpr int U = 8;
        for (int64_t at = lane * 16; at < bytes; at += 512)
            for (int i0 = 0; i0 < n; i0 += U) {
                uint4 x[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < n && src[i0 + u].entry >= 0)
                        x[u] = *reinterpret_cast<const uint4 *>(codes + src[i0 + u].entry * bytes + at);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < n && src[i0 + u].entry >= 0)
                        *reinterpret_cast<uint4 *>(codes + dst[i0 + u].entry * bytes + at) = x[u];
            }
        for (int h = lane; h < p.H; h += 32)
            for (int i0 = 0; i0 < n; i0 += U) {
                unsigned char x[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < n && src[i0 + u].entry >= 0) x[u] = sc[src[i0 + u].scale + (int64_t)h * p.bs];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u < n && src[i0 + u].entry >= 0) sc[dst[i0 + u].scale + (int64_t)h * p.bs] = x[u];
            }
    }
    // every block has read the length; the last one sets it
    __syncthreads();
    if (tid == 0 && atomicAdd(p.counters + b, 1u) == (unsigned)(p.etiles - 1)) {
        p.len[b] = len + n;
        if (p.blocks_in_use) p.blocks_in_use[b] = (len + n) / p.bs + ((len + n) % p.bs != 0);
        p.counters[b] = 0u;
    }
}

template <typename T, int E> cudaError_t launch_rows(Kv8Params p, bool write, cudaStream_t s) {
    p.etiles = (p.S + E - 1) / E;
    const unsigned grid = (unsigned)row_blocks(p.B, p.S, p.H, E);  // (checked: below 2^31)
    auto go = [&](auto g) {
        constexpr int G = decltype(g)::value;  // 8 values a lane
        if (write) write_kv8_kernel<T, G / 2, E><<<grid, kThreads, 0, s>>>(p);
        else read_kv8_kernel<T, G, E><<<grid, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    };
    if (p.D <= 64) return go(std::integral_constant<int, 8>{});
    if (p.D <= 128) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
}

}  // namespace

int64_t kv8_row_blocks(int32_t B, int32_t S, int32_t H) { return row_blocks(B, S, H, 16); }

int64_t kv8_commit_blocks(int32_t B, int32_t L) {
    return (int64_t)B * (((int64_t)2 * L + kCommitUnits - 1) / kCommitUnits);
}

cudaError_t launch_kv8_rows(const Kv8Params &p, int dtype, bool write, int sms, cudaStream_t s) {
    const bool many = row_blocks(p.B, p.S, p.H, 64) >= 2 * sms;
    if (dtype == SPEC_DTYPE_BF16)
        return many ? launch_rows<__nv_bfloat16, 64>(p, write, s) : launch_rows<__nv_bfloat16, 16>(p, write, s);
    return many ? launch_rows<float, 64>(p, write, s) : launch_rows<float, 16>(p, write, s);
}

cudaError_t launch_kv8_commit(Kv8Params p, cudaStream_t s) {
    p.etiles = p.slots ? (int)kv8_commit_blocks(1, p.L) : 1;
    const size_t smem = (size_t)p.S * 2 * sizeof(Place);  // (S <= 1024: 32 KB)
    commit_kv8_kernel<<<(unsigned)((int64_t)p.B * p.etiles), kCommitThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace specv
