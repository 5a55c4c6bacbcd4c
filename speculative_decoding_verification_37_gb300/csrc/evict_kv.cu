// Eviction from the paged cache by accumulated attention weight
// (spec_evict_kv).
//
// evict_select_kernel, one block per request: the entries kept are the
// protected ones (sinks, newest) and the heaviest others; the threshold is the
// exact need-th largest order key, found by four 8-bit histogram passes, ties
// by index.  The keys stay in shared memory where they fit (48 K entries; read
// from L2 in every pass, 2,304 entries took 14 us).  It writes the list of moves
// (kept entries at or past the budget, evicted ones below it, both ascending),
// moves the weights and positions and sets the lengths.  Bound by its barriers:
// a block per request, four passes of histogram and scan.
//
// evict_move_kernel: the moves' sources lie at or past the budget and their
// destinations below it, so no move can overwrite another's source and all run
// at once, in every layer.  Like the commit, one warp moves up to 16 KiB of a
// token's 2*L units with the bulk-copy engine, through shared memory.  It is a
// programmatic dependent of the selection.  Bound by HBM: 16 requests, 32 layers
// of 2 x 8 heads of 128, from up to 2,304 entries to 2,048, 372 MB both ways in
// 63 us (5.9 TB/s); both kernels 80 us.
#include "attn_params.h"
#include "common.cuh"
#include "kernels.h"
#include "tma.cuh"

namespace specv {
namespace {

constexpr int NT = 1024;
constexpr uint32_t kStage = 16384;
constexpr int kKeysMax = 48 * 1024;      // entries whose keys a block keeps
constexpr unsigned kSafe = 0xffffffffu;  // a protected entry's key (no weight has it: it would be a NaN's)

struct SelectSmem {
    unsigned hist[256];
    unsigned scan[33];
    unsigned long long scan2[33];
    unsigned digit, above;
};

// Pages of n entries; pages may be as large as the table (n + bs - 1 would not fit).
__host__ __device__ constexpr int pages_of(int n, int bs) { return n / bs + (n % bs != 0); }
static_assert(pages_of(2000, 0x7fffffff - 1100) == 1 && pages_of(0x7fffffff - 1100, 0x7fffffff - 1100) == 1 &&
                  pages_of(0, 4) == 0 && pages_of(8, 4) == 2 && pages_of(9, 4) == 3,
              "pages");

// exclusive prefix of v over the block, total in *all; two barriers
__device__ __forceinline__ unsigned long long block_prefix(unsigned long long v, unsigned long long *buf, unsigned long long *all) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    unsigned long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += up;
    }
    __syncthreads();
    if (lane == 31) buf[w] = inc;
    __syncthreads();
    unsigned long long before = 0, total = 0;
    const unsigned long long x = buf[lane];
    unsigned long long y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(kFull, y, o);
        if (lane >= o) y += up;
    }
    before = __shfl_sync(kFull, y - x, w);
    total = __shfl_sync(kFull, y, 31);
    *all = total;
    return before + inc - v;
}

__global__ void __launch_bounds__(NT) evict_select_kernel(EvictParams p, int kept_keys) {
    __shared__ SelectSmem sh;
    extern __shared__ unsigned keys[];  // [kept_keys]
    pdl_launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int len = p.len[b];
    float *weight = p.weight + (int64_t)b * p.wstride;
    int *pos = p.key_pos + (int64_t)b * p.kps;
    const int *table = p.table + (int64_t)b * p.max_blocks;
    int2 *moves = p.moves + (int64_t)b * p.max_moves;
    bool bad = len < 0 || (int64_t)len > (int64_t)p.max_blocks * p.bs;
    if (bad || len <= p.budget) {
        if (tid == 0) {
            p.n_moves[b] = 0;
            if (p.blocks_in_use && !bad) p.blocks_in_use[b] = pages_of(len, p.bs);
            if (bad) {
                if (p.flags) atomicOr(p.flags + b, SPEC_FLAG_BAD_INPUT);
                atomicOr(p.status, SPEC_FLAG_BAD_INPUT);
            }
        }
        return;
    }
    int newest = -1;
    for (int i = tid; i < pages_of(len, p.bs); i += NT) {
        const int blk = table[i];
        bad = bad || blk < 0 || (int64_t)blk >= p.nb;
    }
    for (int c = tid; c < len; c += NT) {
        const int q = pos[c];
        const float w = weight[c];
        newest = max(newest, q);
        bad = bad || q < 0 || w != w;
        if (c < kept_keys) keys[c] = fkey(w);
    }
    newest = __reduce_max_sync(kFull, newest);
    if ((tid & 31) == 0) sh.scan[tid >> 5] = (unsigned)newest;
    __syncthreads();
    newest = (int)__reduce_max_sync(kFull, (int)sh.scan[tid & 31]);
    auto safe = [&](int q) { return q < p.sink || q > newest - p.recent; };
    int mine = 0;
    for (int c = tid; c < len; c += NT)
        if (safe(pos[c])) {
            ++mine;
            if (c < kept_keys) keys[c] = kSafe;
        }
    auto key = [&](int c) { return c < kept_keys ? keys[c] : safe(pos[c]) ? kSafe : fkey(weight[c]); };  // (this thread's)
    unsigned long long total;
    block_prefix((unsigned)mine, sh.scan2, &total);
    const int need0 = p.budget - (int)total;
    if (__syncthreads_or(bad || need0 < 0)) {
        if (tid == 0) {
            p.n_moves[b] = 0;
            if (p.blocks_in_use) p.blocks_in_use[b] = pages_of(len, p.bs);
            if (p.flags) atomicOr(p.flags + b, SPEC_FLAG_BAD_INPUT);
            atomicOr(p.status, SPEC_FLAG_BAD_INPUT);
        }
        return;
    }
    // the need0-th largest order key among the others; with need0 == 0 nothing
    // of theirs is kept
    unsigned prefix = 0, need = (unsigned)need0;
    for (int shift = 24; shift >= 0 && need0 > 0; shift -= 8) {
        if (tid < 256) sh.hist[tid] = 0;
        __syncthreads();
        for (int c = tid; c < len; c += NT) {
            const unsigned k = key(c);
            if (k == kSafe) continue;
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&sh.hist[(k >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid < 32) {  // digits from the top: lane 0 holds 255..248
            unsigned s = 0;
            for (int i = 0; i < 8; ++i) s += sh.hist[255 - (tid * 8 + i)];
            unsigned inc = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned up = __shfl_up_sync(kFull, inc, o);
                if (tid >= o) inc += up;
            }
            unsigned above = inc - s;
            if (above < need && need <= inc) {
                for (int i = 0; i < 8; ++i) {
                    const unsigned n = sh.hist[255 - (tid * 8 + i)];
                    if (above + n >= need) {
                        sh.digit = 255 - (tid * 8 + i);
                        sh.above = above;
                        break;
                    }
                    above += n;
                }
            }
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        need -= sh.above;
    }
    // `need` entries equal to the threshold are kept, lowest index first
    unsigned long long ties = 0, lists = 0;
    for (int c0 = 0; c0 < len; c0 += NT) {
        const int c = c0 + tid;
        const bool in = c < len;
        const unsigned k = in ? key(c) : 0u;
        const bool sf = in && k == kSafe;
        const bool eq = in && !sf && need0 > 0 && k == prefix;
        const unsigned long long tie = ties + block_prefix(eq, sh.scan2, &total);
        ties += total;
        const bool kept = sf || (in && !sf && need0 > 0 && (k > prefix || (eq && tie < need)));
        const bool hole = in && !kept && c < p.budget, fill = kept && c >= p.budget;
        const unsigned long long at =
            lists + block_prefix(((unsigned long long)hole << 32) | (unsigned long long)fill, sh.scan2, &total);
        lists += total;
        if (hole) moves[at >> 32].y = c;
        if (fill) moves[at & 0xffffffffull].x = c;
    }
    const int n = (int)(lists & 0xffffffffull);
    __syncthreads();
    for (int i = tid; i < n; i += NT) {
        const int2 m = moves[i];
        weight[m.y] = weight[m.x];
        pos[m.y] = pos[m.x];
    }
    __syncthreads();
    for (int c = p.budget + tid; c < len; c += NT) {
        weight[c] = 0.0f;
        pos[c] = 0;
    }
    if (tid == 0) {
        p.n_moves[b] = n;
        p.len[b] = p.budget;
        if (p.blocks_in_use) p.blocks_in_use[b] = pages_of(p.budget, p.bs);
    }
}

__global__ void __launch_bounds__(32) evict_move_kernel(EvictParams p, CommitGeom geo) {
    __shared__ __align__(128) unsigned char stage[kStage];
    __shared__ __align__(8) unsigned long long bar;
    if (threadIdx.x != 0) return;
    pdl_wait_primary();
    const int grp = blockIdx.x, b = blockIdx.y;
    const int n = p.n_moves[b];
    if ((int)blockIdx.z >= n) return;
    const int *table = p.table + (int64_t)b * p.max_blocks;
    const int64_t unit = p.unit_bytes, plane = p.nb * p.bs * unit;
    const int k0 = grp * geo.upp, k1 = geo.ppu > 1 ? k0 + 1 : min(2 * p.L, k0 + geo.upp);
    auto piece = [&](int k, int64_t &at, uint32_t &bytes) {
        const int lk = k / geo.ppu, sub = k - lk * geo.ppu;
        bytes = (uint32_t)min((int64_t)kStage, unit - (int64_t)sub * kStage);
        at = lk * plane + (int64_t)sub * kStage;
    };
    auto entry = [&](int c) { return ((int64_t)table[c / p.bs] * p.bs + c % p.bs) * unit; };
    uint32_t total = 0;
    for (int k = k0; k < k1; ++k) {
        int64_t at;
        uint32_t bytes;
        piece(k, at, bytes);
        total += bytes;
    }
    mbar_init(&bar, 1);
    fence_barrier_init();
    unsigned phase = 0;
    for (int i = blockIdx.z; i < n; i += gridDim.z, phase ^= 1u) {
        const int2 m = p.moves[(int64_t)b * p.max_moves + i];
        const char *src = p.cache + entry(m.x);
        char *dst = p.cache + entry(m.y);
        bulk_wait_read();  // the stage's last stores have been read
        mbar_arrive_expect_tx(&bar, total);
        uint32_t so = 0;
        for (int k = k0; k < k1; ++k) {
            int64_t at;
            uint32_t bytes;
            piece(k, at, bytes);
            bulk_g2s(stage + so, src + at, bytes, &bar);
            so += bytes;
        }
        if (!mbar_wait_bounded(&bar, phase)) {
            const bool drained = mbar_drain(&bar, phase);
            bulk_wait_read();
            if (drained) mbar_inval(&bar);
            if (p.flags) atomicOr(p.flags + b, SPEC_FLAG_TIMEOUT);
            atomicOr(p.status, SPEC_FLAG_TIMEOUT);
            return;
        }
        so = 0;
        for (int k = k0; k < k1; ++k) {
            int64_t at;
            uint32_t bytes;
            piece(k, at, bytes);
            bulk_s2g(dst + at, stage + so, bytes);
            so += bytes;
        }
        bulk_commit();
    }
    bulk_wait_read();
    mbar_inval(&bar);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t s) {
    const int64_t capacity = (int64_t)p.max_blocks * p.bs;
    const int kept = capacity < kKeysMax ? (int)capacity : kKeysMax;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
    if (e != cudaSuccess) return e;
    evict_select_kernel<<<(unsigned)p.B, NT, (size_t)kept * 4, s>>>(p, kept);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.max_moves == 0) return e;
    const CommitGeom geo = commit_geometry(p.L, p.unit_bytes);
    // about 13 stages fit an SM; blocks past a request's moves leave at once
    int64_t z = ((int64_t)sms * 13 + (int64_t)geo.groups * p.B - 1) / ((int64_t)geo.groups * p.B);
    if (z > p.max_moves) z = p.max_moves;
    if (z > 1024) z = 1024;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)geo.groups, (unsigned)p.B, (unsigned)z);
    cfg.blockDim = dim3(32);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p, geo);
}

}  // namespace specv
