// Internal interface of the operators around the paged cache: attention, entry
// weights, eviction (api_attention.cu and their kernels).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace specv {

int report_cuda_error(cudaError_t e);  // SPEC_OK, or SPEC_ERR_CUDA with the text kept
int device_sms();                      // of the current device

// n / d for n < 2^31: (n * mul) >> shift, mul = ceil(2^(31+s) / d), 2^s >= d.
struct FastDiv {
    unsigned mul, shift;
};
inline FastDiv make_fast_div(unsigned d) {
    unsigned s = 0;
    while ((1ull << s) < d) ++s;
    return FastDiv{(unsigned)(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}
__host__ __device__ inline unsigned fast_div(unsigned n, FastDiv f) {
    return (unsigned)(((unsigned long long)n * f.mul) >> f.shift);
}

struct ScoreArgs {
    float scale, cap, cap_arg;  // cap_arg = 2 log2(e) / cap
    bool bias;
};

constexpr int kAttnThreadsMax = 256;
constexpr int kAttnSmsMax = 160;     // grids are sized for at most this many SMs
constexpr int kAttnSlotRows = 128;   // rows of partial results per SM and slot; twice that with a shared prefix
constexpr int kAttnBlocksMax = kAttnSmsMax * 8;

struct SplitItem {                // an item that goes on past the block it begins in
    int blocks;                   // how many it lies in; 0: there is none
    int b, h, rt, ok;
};

struct AttnParams {
    int B, S, Hq, H, G, D, bs, max_blocks, W;
    int64_t nb;
    FastDiv bs_div;
    const void *q;
    int64_t qsb, qss, qsh;
    const void *kc, *vc;          // the layer's planes [nb][bs][H][D]
    const void *tk, *tv;          // the layer's candidates of request 0, or null (in place)
    int64_t tsb;                  // elements between two requests' candidates
    const void *temp_base;        // [B][layers][2][S][H][D]
    int layers, layer;
    const int *table, *len;
    const uint32_t *mask;
    const int *pos, *key_pos;
    int64_t kps;
    const int *first;
    const float *slopes;
    ScoreArgs score;
    int window;
    int P;                        // shared entries
    const int *stable;            // their blocks
    int mode;                     // 0: each request's own keys; 1: the shared prefix, all requests'
                                  // rows; 2: the committed entries (weights)
    const int *slots, *n_slots;   // mode 2: the committed candidates
    int slots_stride;
    int min_share;                // tiles a block takes at least
    int box;                      // rows of a page copied at once (0: row by row)
    void *out;
    float *lse;
    unsigned *flags, *status;
    unsigned *counters;           // [block] arrivals at the split item that begins in it; zero between calls
    SplitItem *split;             // [block]
    float *part;                  // partial results [block][2][rows][D + 2]
    float *pre_o, *pre_lse;       // shared part: normalised rows and log2 sums
};
// joins what launch_attn_tc left split (it calls it; bf16); rt_rows: queries of an item
cudaError_t launch_attn_join(const AttnParams &p, int rt_rows, int blocks, cudaStream_t s);
cudaError_t launch_attn_simt(const AttnParams &p, int sms, cudaStream_t s);  // f32
cudaError_t launch_attn_mma(const AttnParams &p, int sms, cudaStream_t s);  // bf16
// bf16, keys in boxes: p.box from attn_tc_box (0: this kernel does not take the call)
int attn_tc_box(const AttnParams &p);
cudaError_t launch_attn_tc(const AttnParams &p, int sms, cudaStream_t s);

struct WeightsParams {
    AttnParams a;                 // q, cache, tables, score (P: entries left out)
    const float *lse_in;
    int *key_pos_out;
    float *weight;
    int64_t wstride;
};
cudaError_t launch_weights(const WeightsParams &p, int dtype, int sms, cudaStream_t s);
// bf16 with p.a.box set (attn_tc_box); 0 candidates a pass: this kernel does not take the call
int weights_tc_per_pass(const AttnParams &p);
cudaError_t launch_weights_tc(const WeightsParams &p, int per_pass, int sms, cudaStream_t s);

struct EvictParams {
    int B, L, bs, max_blocks, unit_bytes, budget, sink, recent, max_moves;
    char *cache;
    int64_t nb;
    const int *table;
    int *len;
    float *weight;
    int64_t wstride;
    int *key_pos;
    int64_t kps;
    int *blocks_in_use;
    unsigned *flags, *status;
    int *n_moves;                 // [B]
    int2 *moves;                  // [B][max_moves] (from, to) entries
};
cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t s);
// workspace layouts (null base: the size alone)
size_t attn_ws_layout(int32_t B, int32_t n, int32_t D, bool shared, void *base, AttnParams *p);
size_t evict_ws_layout(int32_t B, int32_t budget, int32_t capacity, void *base, EvictParams *p);


}  // namespace specv
