// The 8-bit cache's writer, reader and the commit of a tree's path
// (spec_write_kv_q8, spec_read_kv_q8, spec_commit_kv_q8); its numbers: kv8.cuh.
//
// Writing and reading: a block has 16 entries and up to 32 heads of K or V, a group
// of lanes a row, 8 values a lane; a row's largest magnitude is a few shuffles.
// The rows' exponents lie a head's next to each other, so that attention reads a
// page's in one piece: they pass through shared memory and leave 16 bytes a head.
// Bound by HBM.
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

constexpr int kEntries = 16, kHeads = 32, kThreads = 256;

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

// 8 values of a row
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = ld_nc16(p); }
    __device__ __forceinline__ void values(float *x) const { unpack<__nv_bfloat16>(v, x); }
};
template <> struct Raw8<float> {
    uint4 v, w;
    __device__ __forceinline__ void load(const float *p) {
        v = ld_nc16(p);
        w = ld_nc16(p + 4);
    }
    __device__ __forceinline__ void values(float *x) const {
        unpack<float>(v, x);
        unpack<float>(w, x + 4);
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
// Blocks: K/V fastest, then head chunks, entries, requests.
__device__ __forceinline__ Tile tile_of(const Kv8Params &p) {
    Tile t;
    int64_t i = blockIdx.x;
    t.kv = (int)(i & 1);
    i >>= 1;
    const int chunks = (p.H + kHeads - 1) / kHeads;
    t.h0 = (int)(i % chunks) * kHeads;
    i /= chunks;
    t.heads = min(kHeads, p.H - t.h0);
    t.e0 = (int)(i % p.etiles) * kEntries;
    t.b = (int)(i / p.etiles);
    return t;
}

// G: lanes of a row
template <typename T, int G> __global__ void __launch_bounds__(kThreads) write_kv8_kernel(Kv8Params p) {
    __shared__ Place place[kEntries];
    __shared__ unsigned char scale[kHeads][kEntries];
    const Tile t = tile_of(p);
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
    const int entries = min(kEntries, n - t.e0);
    if (entries <= 0) return;
    if (tid < entries) place[tid] = place_of(p, t.b, len + t.e0 + tid);
    __syncthreads();
    constexpr int NG = kThreads / G, U = 4;
    const int d = (tid % G) * 8, rows = entries * t.heads;
    const bool in = d < p.D;
    const T *src = static_cast<const T *>(t.kv ? p.v : p.k) + t.b * p.sb[t.kv];
    unsigned char *codes = p.codes + (t.kv ? p.plane : 0);
    for (int base = 0; base < rows; base += NG * U) {  // (every lane takes part in the shuffles)
        const int r0 = base + tid / G;
        Raw8<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * NG, e = r / t.heads, h = t.h0 + r - e * t.heads;
            if (r < rows && in) raw[u].load(src + (t.e0 + e) * p.ss[t.kv] + h * p.sh[t.kv] + d);
        }
        float top[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            top[u] = 0.0f;
            if (r0 + u * NG < rows && in) {
                float x[8];
                raw[u].values(x);
                bool odd = false;  // (fmaxf leaves a NaN out)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    top[u] = fmaxf(top[u], fabsf(x[i]));
                    odd = odd || x[i] != x[i];
                }
                if (odd) top[u] = INFINITY;
            }
#pragma unroll
            for (int q = G / 2; q > 0; q >>= 1) top[u] = fmaxf(top[u], __shfl_xor_sync(kFull, top[u], q));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * NG;
            if (r >= rows) break;
            const int e = r / t.heads, h = r - e * t.heads;
            const unsigned s = kv8_scale(top[u]);
            if (d == 0) scale[h][e] = (unsigned char)s;
            if (!in || place[e].entry < 0) continue;
            uint2 c = make_uint2(0u, 0u);
            if (s != 255u) {
                float x[8];
                raw[u].values(x);
                const float f = kv8_inverse(s);
                c.x = kv8_code2(x[0] * f, x[1] * f) | kv8_code2(x[2] * f, x[3] * f) << 16;
                c.y = kv8_code2(x[4] * f, x[5] * f) | kv8_code2(x[6] * f, x[7] * f) << 16;
            }
            *reinterpret_cast<uint2 *>(codes + (place[e].entry * p.H + t.h0 + h) * p.D + d) = c;
        }
    }
    __syncthreads();
    unsigned char *sc = p.scale + (t.kv ? p.splane : 0);
    for (int i = tid; i < t.heads * kEntries; i += kThreads) {
        const int h = i / kEntries, e = i - h * kEntries;
        if (e < entries && place[e].entry >= 0) sc[place[e].scale + (int64_t)(t.h0 + h) * p.bs] = scale[h][e];
    }
}

template <typename T, int G> __global__ void __launch_bounds__(kThreads) read_kv8_kernel(Kv8Params p) {
    __shared__ Place place[kEntries];
    __shared__ float power[kHeads][kEntries];
    const Tile t = tile_of(p);
    const int tid = threadIdx.x;
    const int start = p.start ? p.start[t.b] : 0, n = p.count ? p.count[t.b] : p.S;
    const bool good = start >= 0 && n >= 0 && n <= p.S && (int64_t)start + n <= (int64_t)p.max_blocks * p.bs;
    if (!good && t.e0 == 0 && t.h0 == 0 && t.kv == 0 && tid == 0) {
        if (p.flags) atomicOr(p.flags + t.b, SPEC_FLAG_BAD_INPUT);
        atomicOr(p.status, SPEC_FLAG_BAD_INPUT);
    }
    const int entries = min(kEntries, p.S - t.e0), held = good ? min(entries, n - t.e0) : 0;
    if (tid < entries) place[tid] = tid < held ? place_of(p, t.b, start + t.e0 + tid) : Place{-1, 0};
    __syncthreads();
    const unsigned char *sc = p.scale + (t.kv ? p.splane : 0), *codes = p.codes + (t.kv ? p.plane : 0);
    for (int i = tid; i < t.heads * kEntries; i += kThreads) {
        const int h = i / kEntries, e = i - h * kEntries;
        if (e < entries && place[e].entry >= 0)
            power[h][e] = kv8_power(__ldg(sc + place[e].scale + (int64_t)(t.h0 + h) * p.bs));
    }
    __syncthreads();
    constexpr int NG = kThreads / G, U = 4;
    const int d = (tid % G) * 8, rows = entries * t.heads;
    if (d >= p.D) return;
    T *out = static_cast<T *>(t.kv ? p.out_v : p.out_k) + ((int64_t)t.b * p.S + t.e0) * p.H * p.D;
    for (int r0 = tid / G; r0 < rows; r0 += NG * U) {
        uint2 c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * NG, e = r / t.heads, h = t.h0 + r - e * t.heads;
            c[u] = make_uint2(0u, 0u);
            if (r < rows && place[e].entry >= 0)
                c[u] = __ldg(reinterpret_cast<const uint2 *>(codes + (place[e].entry * p.H + h) * p.D + d));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * NG;
            if (r >= rows) continue;
            const int e = r / t.heads, h = r - e * t.heads;
            const float f = place[e].entry >= 0 ? power[h][e] : 0.0f;
            const float4 a = kv8_value4(c[u].x), b = kv8_value4(c[u].y);
            const float x[8] = {a.x * f, a.y * f, a.z * f, a.w * f, b.x * f, b.y * f, b.z * f, b.w * f};
            store8(out + ((int64_t)e * p.H + t.h0 + h) * p.D + d, x);
        }
    }
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

template <typename T> cudaError_t launch_rows(const Kv8Params &p, bool write, cudaStream_t s) {
    const int64_t grid = kv8_row_blocks(p.B, p.S, p.H);  // (checked: below 2^31)
    auto go = [&](auto g) {
        constexpr int G = decltype(g)::value;
        if (write) write_kv8_kernel<T, G><<<(unsigned)grid, kThreads, 0, s>>>(p);
        else read_kv8_kernel<T, G><<<(unsigned)grid, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    };
    if (p.D <= 64) return go(std::integral_constant<int, 8>{});
    if (p.D <= 128) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
}

}  // namespace

int64_t kv8_row_blocks(int32_t B, int32_t S, int32_t H) {
    return (int64_t)B * ((S + kEntries - 1) / kEntries) * ((H + kHeads - 1) / kHeads) * 2;
}

int64_t kv8_commit_blocks(int32_t B, int32_t L) {
    return (int64_t)B * (((int64_t)2 * L + kCommitUnits - 1) / kCommitUnits);
}

cudaError_t launch_kv8_rows(Kv8Params p, int dtype, bool write, cudaStream_t s) {
    p.etiles = (p.S + kEntries - 1) / kEntries;
    return dtype == SPEC_DTYPE_BF16 ? launch_rows<__nv_bfloat16>(p, write, s) : launch_rows<float>(p, write, s);
}

cudaError_t launch_kv8_commit(Kv8Params p, cudaStream_t s) {
    p.etiles = p.slots ? (int)kv8_commit_blocks(1, p.L) : 1;
    const size_t smem = (size_t)p.S * 2 * sizeof(Place);  // (S <= 1024: 32 KB)
    commit_kv8_kernel<<<(unsigned)((int64_t)p.B * p.etiles), kCommitThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace specv
