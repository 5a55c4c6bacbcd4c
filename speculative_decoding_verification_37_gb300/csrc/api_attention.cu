// C ABI of the operators around the paged cache: argument checks, workspace
// layouts, launches (spec_verify_attention, spec_attention_weights,
// spec_evict_kv).
#include <cmath>

#include "attn_params.h"
#include "kernels.h"
#include "spec_verify.h"

using namespace specv;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The checks and parameters the two calls that score queries share.
template <typename A> int scored_call(const A *a, AttnParams &p) {
    if (a->B < 0 || a->B > 32768 || a->S < 1 || a->S > SPEC_ATTENTION_MAX_S || a->H < 1 || a->Hq < 1 ||
        a->Hq % a->H != 0 || a->D < 1 || a->L < 1 || a->layer < 0 || a->layer >= a->L)
        return SPEC_ERR_INVALID_ARG;
    if (a->dtype != SPEC_DTYPE_BF16 && a->dtype != SPEC_DTYPE_F32) return SPEC_ERR_INVALID_ARG;
    if (a->block_size < 1 || a->max_blocks < 1 || a->num_blocks < 1) return SPEC_ERR_INVALID_ARG;
    if (!std::isfinite(a->scale) || !(a->softcap >= 0.0f) || a->window < 0 || a->shared_len < 0)
        return SPEC_ERR_INVALID_ARG;
    const float cap_arg = a->softcap > 0.0f ? (float)(2.0 * 1.4426950408889634074 / (double)a->softcap) : 0.0f;
    if (!std::isfinite(a->softcap) || !std::isfinite(cap_arg) || !std::isfinite(a->scale * cap_arg))
        return SPEC_ERR_INVALID_ARG;
    const int64_t e = a->dtype == SPEC_DTYPE_BF16 ? 2 : 4;
    if (a->D > SPEC_ATTENTION_MAX_D || a->D * e % 16 != 0) return SPEC_ERR_UNSUPPORTED;
    // the bf16 kernels' tanh is exact to a few 2^-24 of the cap: 2^-12 of a score at 1024
    if (a->dtype == SPEC_DTYPE_BF16 && a->softcap > 1024.0f) return SPEC_ERR_UNSUPPORTED;
    const int64_t capacity = (int64_t)a->max_blocks * a->block_size;
    if (capacity > 0x7fffffffLL - 2 * SPEC_ATTENTION_MAX_S || a->Hq > 65535) return SPEC_ERR_UNSUPPORTED;
    if (a->shared_len > capacity) return SPEC_ERR_INVALID_ARG;
    if (a->key_pos && a->key_pos_stride < capacity) return SPEC_ERR_INVALID_ARG;
    if (a->B == 0) return SPEC_OK;
    if (!a->q || !a->cache || !a->block_table || !a->committed_len) return SPEC_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->cache, 16) || a->q_stride_b * e % 16 || a->q_stride_s * e % 16 ||
        a->q_stride_h * e % 16)
        return SPEC_ERR_INVALID_ARG;
    p = AttnParams{};
    p.B = a->B;
    p.S = a->S;
    p.Hq = a->Hq;
    p.H = a->H;
    p.G = a->Hq / a->H;
    p.D = a->D;
    p.bs = a->block_size;
    p.bs_div = make_fast_div((unsigned)a->block_size);
    p.max_blocks = a->max_blocks;
    p.W = (a->S + 31) / 32;
    p.nb = a->num_blocks;
    p.q = a->q;
    p.qsb = a->q_stride_b;
    p.qss = a->q_stride_s;
    p.qsh = a->q_stride_h;
    const int64_t plane = a->num_blocks * a->block_size * a->H * a->D * e;
    p.kc = static_cast<const char *>(a->cache) + plane * 2 * a->layer;
    p.vc = static_cast<const char *>(p.kc) + plane;
    p.table = a->block_table;
    p.len = a->committed_len;
    p.pos = a->pos;
    p.key_pos = a->key_pos;
    p.kps = a->key_pos_stride;
    p.first = a->first_pos;
    p.slopes = a->slopes;
    p.score = ScoreArgs{a->scale, a->softcap, cap_arg, a->slopes != nullptr};
    p.window = a->window;
    p.layers = a->L;
    p.layer = a->layer;
    p.P = a->shared_len;
    p.flags = a->flags;
    return SPEC_OK;
}

}  // namespace

namespace specv {

size_t attn_ws_layout(int32_t B, int32_t n, int32_t D, bool shared, void *base, AttnParams *p) {
    size_t off = kWsHeader;
    const size_t o_split = off;
    off += ws_align(kAttnBlocksMax * sizeof(SplitItem));
    const size_t o_cnt = off;
    off += ws_align(kAttnBlocksMax * sizeof(unsigned));
    static_assert(kWsHeader + kAttnBlocksMax * (sizeof(SplitItem) + sizeof(unsigned)) + 2 * 256 <= SPEC_WS_ZEROED,
                  "the counters lie in the zeroed part");
    const size_t o_part = off;
    off += ws_align((size_t)kAttnSmsMax * 2 * kAttnSlotRows * (shared ? 2 : 1) * ((size_t)D + 2) * sizeof(float));
    const size_t o_pre = off;
    if (shared) off += ws_align((size_t)B * n * D * sizeof(float));
    const size_t o_lse = off;
    if (shared) off += ws_align((size_t)B * n * sizeof(float));
    if (p) {
        char *c = static_cast<char *>(base);
        p->status = reinterpret_cast<unsigned *>(c);
        p->split = reinterpret_cast<SplitItem *>(c + o_split);
        p->counters = reinterpret_cast<unsigned *>(c + o_cnt);
        p->part = reinterpret_cast<float *>(c + o_part);
        p->pre_o = reinterpret_cast<float *>(c + o_pre);
        p->pre_lse = reinterpret_cast<float *>(c + o_lse);
    }
    return off;
}

// A request moves at most as many entries as lie past the budget, or below it.
size_t evict_ws_layout(int32_t B, int32_t budget, int32_t capacity, void *base, EvictParams *p) {
    const int32_t over = capacity > budget ? capacity - budget : 0;
    const int32_t most = over < budget ? over : budget;
    size_t off = kWsHeader;
    const size_t o_n = off;
    off += ws_align((size_t)B * sizeof(int));
    const size_t o_m = off;
    off += ws_align((size_t)B * most * sizeof(int2));
    if (p) {
        char *c = static_cast<char *>(base);
        p->status = reinterpret_cast<unsigned *>(c);
        p->n_moves = reinterpret_cast<int *>(c + o_n);
        p->moves = reinterpret_cast<int2 *>(c + o_m);
        p->max_moves = most;
    }
    return off;
}

}  // namespace specv

extern "C" int spec_verify_attention(const SpecAttentionArgs *a, void *workspace, size_t ws_bytes, void *stream) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    AttnParams p;
    const int chk = scored_call(a, p);
    if (chk != SPEC_OK || a->B == 0) return chk;
    if (!a->out || !aligned(a->out, 16) || (a->temp_kv && !aligned(a->temp_kv, 16))) return SPEC_ERR_INVALID_ARG;
    if (a->shared_len > 0 && (!a->shared_table || a->key_pos)) return SPEC_ERR_INVALID_ARG;
    const int kind = a->shared_len > 0 ? SPEC_WS_ATTENTION_SHARED : SPEC_WS_ATTENTION;
    if ((int64_t)a->S * a->Hq > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, 256) ||
        ws_bytes < spec_workspace_bytes(kind, a->B, a->S * a->Hq, a->D))
        return SPEC_ERR_INVALID_ARG;
    attn_ws_layout(a->B, a->S * a->Hq, a->D, a->shared_len > 0, workspace, &p);
    const int64_t e = a->dtype == SPEC_DTYPE_BF16 ? 2 : 4;
    if (a->temp_kv) {
        const int64_t one = (int64_t)a->S * a->H * a->D * e;  // one layer's K or V of a request
        p.tk = static_cast<const char *>(a->temp_kv) + one * 2 * a->layer;
        p.tv = static_cast<const char *>(p.tk) + one;
        p.tsb = (int64_t)a->L * 2 * a->S * a->H * a->D;
        p.temp_base = a->temp_kv;
    }
    p.mask = a->tree_mask;
    p.stable = a->shared_table;
    p.out = a->out;
    p.lse = a->lse;
    p.min_share = 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int sms = device_sms();
    auto launch = [&](AttnParams &x) {
        if (a->dtype != SPEC_DTYPE_BF16) return launch_attn_simt(x, sms, s);
        x.box = attn_tc_box(x);
        return x.box ? launch_attn_tc(x, sms, s) : launch_attn_mma(x, sms, s);
    };
    if (a->shared_len > 0) {
        AttnParams q = p;
        q.mode = 1;
        const cudaError_t err = launch(q);
        if (err != cudaSuccess) return report_cuda_error(err);
    }
    return report_cuda_error(launch(p));
}

extern "C" int spec_attention_weights(const SpecWeightsArgs *a, void *workspace, size_t ws_bytes, void *stream) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    WeightsParams w;
    const int chk = scored_call(a, w.a);
    if (chk != SPEC_OK || a->B == 0) return chk;
    if (!a->lse || !a->n_slots || !a->weight) return SPEC_ERR_INVALID_ARG;
    if (a->slots && a->slots_stride < a->S) return SPEC_ERR_INVALID_ARG;
    if (a->weight_stride < (int64_t)a->max_blocks * a->block_size) return SPEC_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || ws_bytes < spec_workspace_bytes(SPEC_WS_COMMIT, a->B, 0, 0))
        return SPEC_ERR_INVALID_ARG;
    w.a.status = static_cast<unsigned *>(workspace);
    w.a.mode = 2;
    w.a.min_share = 1;
    w.a.slots = a->slots;
    w.a.n_slots = a->n_slots;
    w.a.slots_stride = a->slots_stride;
    w.lse_in = a->lse;
    w.key_pos_out = a->key_pos;
    w.weight = a->weight;
    w.wstride = a->weight_stride;
    return report_cuda_error(launch_weights(w, a->dtype, device_sms(), static_cast<cudaStream_t>(stream)));
}

extern "C" int spec_evict_kv(const SpecEvictArgs *a, void *workspace, size_t ws_bytes, void *stream) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    if (a->B < 0 || a->B > 32768 || a->L < 1 || a->H < 1 || a->D < 1 || a->block_size < 1 || a->num_blocks < 1 ||
        a->max_blocks < 1)
        return SPEC_ERR_INVALID_ARG;
    if (a->elem_bytes != 1 && a->elem_bytes != 2 && a->elem_bytes != 4) return SPEC_ERR_INVALID_ARG;
    if (a->budget < 1 || a->sink < 0 || a->recent < 0 || (int64_t)a->sink + a->recent > a->budget)
        return SPEC_ERR_INVALID_ARG;
    const int64_t unit = (int64_t)a->H * a->D * a->elem_bytes, capacity = (int64_t)a->max_blocks * a->block_size;
    if (unit % 16 != 0 || unit > (1 << 20) || capacity > 0x7fffffffLL - 1024) return SPEC_ERR_UNSUPPORTED;
    if (a->weight_stride < capacity || a->key_pos_stride < capacity) return SPEC_ERR_INVALID_ARG;
    if (a->B == 0) return SPEC_OK;
    if (!a->cache || !aligned(a->cache, 16) || !a->block_table || !a->committed_len || !a->weight || !a->key_pos)
        return SPEC_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        ws_bytes < spec_workspace_bytes(SPEC_WS_EVICT, a->B, a->budget, (int32_t)capacity))
        return SPEC_ERR_INVALID_ARG;
    EvictParams p = {};
    evict_ws_layout(a->B, a->budget, (int32_t)capacity, workspace, &p);
    p.B = a->B;
    p.L = a->L;
    p.bs = a->block_size;
    p.max_blocks = a->max_blocks;
    p.unit_bytes = (int)unit;
    p.budget = a->budget;
    p.sink = a->sink;
    p.recent = a->recent;
    p.cache = static_cast<char *>(a->cache);
    p.nb = a->num_blocks;
    p.table = a->block_table;
    p.len = a->committed_len;
    p.weight = a->weight;
    p.wstride = a->weight_stride;
    p.key_pos = a->key_pos;
    p.kps = a->key_pos_stride;
    p.blocks_in_use = a->blocks_in_use;
    p.flags = a->flags;
    return report_cuda_error(launch_evict(p, device_sms(), static_cast<cudaStream_t>(stream)));
}
