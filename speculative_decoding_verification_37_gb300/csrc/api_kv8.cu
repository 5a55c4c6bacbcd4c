// C ABI of the 8-bit cache's writer, reader and commit: argument checks, launches
// (spec_write_kv_q8, spec_read_kv_q8, spec_commit_kv_q8).
#include "attn_params.h"
#include "kernels.h"
#include "spec_verify.h"

using namespace specv;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The checks and parameters the three calls share.  (A request without entries
// needs none of the pointers.)
template <typename A> int kv8_call(const A *a, void *workspace, size_t ws_bytes, int layer, Kv8Params &p) {
    if (a->B < 0 || a->B > 32768 || a->S < 1 || a->H < 1 || a->D < 1 || a->L < 1 || layer < 0 || layer >= a->L ||
        a->block_size < 1 || a->max_blocks < 1 || a->num_blocks < 1)
        return SPEC_ERR_INVALID_ARG;
    const int64_t capacity = (int64_t)a->max_blocks * a->block_size;
    if (a->D % 16 != 0 || a->D > SPEC_ATTENTION_MAX_D || a->H > 65535 || a->S > (1 << 30) ||
        capacity > 0x7fffffffLL - 2 * SPEC_ATTENTION_MAX_S)
        return SPEC_ERR_UNSUPPORTED;
    if (a->B == 0) return SPEC_OK;
    if (!a->codes || !aligned(a->codes, 16) || !a->scale || !a->block_table) return SPEC_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || ws_bytes < spec_workspace_bytes(SPEC_WS_KV8, a->B, 0, 0))
        return SPEC_ERR_INVALID_ARG;
    p = Kv8Params{};
    p.B = a->B;
    p.S = a->S;
    p.L = a->L;
    p.H = a->H;
    p.D = a->D;
    p.bs = a->block_size;
    p.bs_div = make_fast_div((unsigned)a->block_size);
    p.max_blocks = a->max_blocks;
    p.nb = a->num_blocks;
    p.splane = a->num_blocks * a->block_size * a->H;
    p.plane = p.splane * a->D;
    p.codes = static_cast<unsigned char *>(const_cast<void *>(static_cast<const void *>(a->codes))) + p.plane * 2 * layer;
    p.scale = const_cast<unsigned char *>(a->scale) + p.splane * 2 * layer;
    p.table = a->block_table;
    p.flags = a->flags;
    p.status = static_cast<unsigned *>(workspace);
    p.counters = reinterpret_cast<unsigned *>(static_cast<char *>(workspace) + kWsHeader);
    return SPEC_OK;
}

}  // namespace

extern "C" int spec_write_kv_q8(const SpecWriteKvQ8Args *a, void *workspace, size_t ws_bytes, void *stream) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    if (a->dtype != SPEC_DTYPE_BF16 && a->dtype != SPEC_DTYPE_F32) return SPEC_ERR_INVALID_ARG;
    Kv8Params p;
    const int chk = kv8_call(a, workspace, ws_bytes, a->layer, p);
    if (chk != SPEC_OK || a->B == 0) return chk;
    const int64_t e = a->dtype == SPEC_DTYPE_BF16 ? 2 : 4;
    if (!a->k || !a->v || !aligned(a->k, 16) || !aligned(a->v, 16) || !a->committed_len) return SPEC_ERR_INVALID_ARG;
    if (a->k_stride_b * e % 16 || a->k_stride_s * e % 16 || a->k_stride_h * e % 16 || a->v_stride_b * e % 16 ||
        a->v_stride_s * e % 16 || a->v_stride_h * e % 16)
        return SPEC_ERR_INVALID_ARG;
    if (kv8_row_blocks(a->B, a->S, a->H) > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
    p.k = a->k;
    p.v = a->v;
    p.sb[0] = a->k_stride_b;
    p.ss[0] = a->k_stride_s;
    p.sh[0] = a->k_stride_h;
    p.sb[1] = a->v_stride_b;
    p.ss[1] = a->v_stride_s;
    p.sh[1] = a->v_stride_h;
    p.start = a->committed_len;
    p.count = a->n_new;
    return report_cuda_error(launch_kv8_rows(p, a->dtype, true, device_sms(), static_cast<cudaStream_t>(stream)));
}

extern "C" int spec_read_kv_q8(const SpecReadKvQ8Args *a, void *workspace, size_t ws_bytes, void *stream) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    if (a->dtype != SPEC_DTYPE_BF16 && a->dtype != SPEC_DTYPE_F32) return SPEC_ERR_INVALID_ARG;
    Kv8Params p;
    const int chk = kv8_call(a, workspace, ws_bytes, a->layer, p);
    if (chk != SPEC_OK || a->B == 0) return chk;
    if (!a->k || !a->v || !aligned(a->k, 16) || !aligned(a->v, 16)) return SPEC_ERR_INVALID_ARG;
    if (kv8_row_blocks(a->B, a->S, a->H) > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
    p.out_k = a->k;
    p.out_v = a->v;
    p.start = a->start;
    p.count = a->count;
    return report_cuda_error(launch_kv8_rows(p, a->dtype, false, device_sms(), static_cast<cudaStream_t>(stream)));
}

extern "C" int spec_commit_kv_q8(const SpecCommitKvQ8Args *a, void *workspace, size_t ws_bytes, void *stream) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    Kv8Params p;
    const int chk = kv8_call(a, workspace, ws_bytes, 0, p);
    if (chk != SPEC_OK) return chk;
    if (a->S > SPEC_ATTENTION_MAX_S) return SPEC_ERR_UNSUPPORTED;
    if (a->B == 0) return SPEC_OK;
    if (!a->n_slots || !a->committed_len || (a->slots && a->slots_stride < a->S)) return SPEC_ERR_INVALID_ARG;
    if (kv8_commit_blocks(a->B, a->L) > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
    p.slots = a->slots;
    p.slots_stride = a->slots_stride;
    p.count = a->n_slots;
    p.len = a->committed_len;
    p.blocks_in_use = a->blocks_in_use;
    return report_cuda_error(launch_kv8_commit(p, static_cast<cudaStream_t>(stream)));
}
